// cp_attn_tree for many rows a request and KV head (trees, longer drafts, chunks): tcgen05.
//
// A unit is one MMA tile of 128 packed rows (single), or two (dual).  Two softmax
// warpgroups (streams) work at a time: of a dual unit each has one tile's rows and both use
// every KV tile of 128 keys; of a single unit both have all rows, and the KV tiles alternate
// between them, so that one stream's softmax runs under the other's products, too.
//   warps 0-7    softmax, one row a thread: S from TMEM, mask (tiles with new keys only),
//                online softmax in base 2 with a lazily moved maximum, P back to TMEM in 16
//                bits; at a piece's end O / l from TMEM to the output, or to the workspace
//                where the unit is cut.  A single unit's two halves are joined there, each
//                stream half of the columns.
//   warps 8, 9   producers of the K and the V tiles: a lane looks up a page, a tile ahead,
//                and starts its TMA copies; one ring of tiles in the order of use that runs
//                across piece ends.
//   warp 10      MMA issuer: O += P V and the next S = Q K^T of one stream, then
//                of the other.
//   warp 11      query rows to shared memory, over codes turned to f16 (the first piece's by
//                the softmax warps); walks the share.
//   warps 12-19  (e4m3 cache) codes to f16 tiles, as in attn_shared.cu.
// Every wait is bounded; warp 11 walks the block's share and the others read its pieces from
// a ring (see attn_tree.cuh).
//
// Value rows behind the last key, and (among new keys) rows with an infinity or a NaN, become
// zeros in shared memory before their product: 0 * NaN is NaN, so that masking P alone
// would not keep them from the rows that do not see them.  A row that does see one becomes
// NaN by its sum.
//
// Codes of cached keys, which all rows of a request see, are turned to f16 with one exponent a tile.
// In a tile with new keys that would let the scale of a key that a row does not see take the bits
// of those that it sees: there codes stay as they are, and K's scales go to the scores, V's to the
// weights (softmax_row_scaled; it costs 2 us at a piece's end, e4m3 trees of 26 at d = 64 31.3 -> 33.4 us,
// while the other tiles' code is rid of its masks, e4m3 trees of 64 407 -> 364).
//
// Measured on the device, 32/8 heads, d = 128, 32 requests on up to 16K keys: trees of 32 (single units)
// 209 us, HBM (floor 193); trees of 64 (dual) 257 us at 2.07 GHz, 273 at the 1.8 GHz of a steady run
// (floor 194): the tensor pipe is active 60 % of the cycles, a stream's chain S -> softmax -> P ->
// P V is what bounds them.  Over codes 262 and 364 us (floors 100 and 130): the same chain with S in
// halves, beside the converters.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "attn_tree_smem.cuh"

namespace cpattn {
namespace {

// The MMAs and commits of ptx.cuh, by the lane with `lead` of a whole warp.
__device__ __forceinline__ void mma_ss_lead(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts_lead(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_commit_lead(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}

// The words of a row's mask that hold the bits of a tile's 128 keys, the first of which is new
// key n (negative: cached keys before it).  Fetched before they are needed.
struct MaskWords {
  uint32_t w[5];
  __device__ __forceinline__ void load(const TreeParams& p, const TreePiece& pc, int node, int n) {
    const int first = n >> 5;  // (rounds down)
#pragma unroll
    for (int x = 0; x < 5; ++x) {
      const int at = first + x;
      w[x] = !p.mask ? ~0u
             : at >= 0 && at < p.words ? (uint32_t)__ldg(p.mask + (long long)(pc.row0 + node) * p.words + at)
                                       : 0u;
    }
  }
  // The keys of the tile that the row sees; limit: the new keys that it may see.
  __device__ __forceinline__ void seen(int n, int limit, uint32_t (&vis)[4]) const {
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int m = n + 32 * x;  // new key of the word's first bit
      uint32_t bits = __funnelshift_r(w[x], w[x + 1], n & 31);
      if (m < 0) bits |= m <= -32 ? ~0u : (1u << -m) - 1u;  // cached keys
      const int count = limit - m;
      vis[x] = count >= 32 ? bits : count <= 0 ? 0u : bits & ((1u << count) - 1u);
    }
  }
};

// A query row of bf16 to f16 times 2^f with 2^f max|q| in [2^14, 2^15).
struct QueryLift {
  float up;
  __device__ __forceinline__ QueryLift(uint32_t largest, int& f) {  // bits of max|q|
    f = min(max(14 - ((int)(largest >> 7) - 127), -126), 126);
    up = exp2_int(f);
  }
  __device__ __forceinline__ uint32_t two(uint32_t v) const {
    return pack_f16x2(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xFFFF0000u) * up);
  }
  __device__ __forceinline__ uint4 operator()(const uint4& v) const {
    return make_uint4(two(v.x), two(v.y), two(v.z), two(v.w));
  }
};

// A barrier of 256 threads; true when all of them say so.
__device__ __forceinline__ bool bar_all(int id, bool all) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
      "bar.red.and.pred q, %1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"((uint32_t)all)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void bar_named(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// O of a warp's rows (one a lane) times f, where a row needs it.
template <int D>
__device__ __forceinline__ void rescale_row(uint32_t o_addr, bool need, float f) {
  if (!__any_sync(0xffffffffu, need)) return;
  const float a = need ? f : 1.f;
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

// S of a tile to P, for the rows of a warp (one a lane): see softmax_tile in attn_shared.cu.
// vis: the keys that the row sees (masked: not all); o_scale: what O is multiplied by besides.
// Over codes S goes through the registers by halves, the first one twice (for the maximum and for
// P): the converters have the registers that a whole row would take.
template <int D, bool QUANT>
__device__ __forceinline__ void softmax_row(uint32_t s_addr, uint32_t o_addr, bool masked, const uint32_t (&vis)[4],
                                            bool has_o, float o_scale, float sl2, float& m_run, float& m_use,
                                            float& l_run) {
  constexpr int kParts = QUANT ? 2 : 1, kCols = BN / kParts;
  float x[kCols];
  auto load = [&](int part) {
    uint32_t v[kCols];
#pragma unroll
    for (int q = 0; q < kCols / 32; ++q) tmem_ld32p(s_addr + part * kCols + q * 32, v + q * 32);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < kCols; ++c) x[c] = __uint_as_float(v[c]);
    if (masked) {
#pragma unroll
      for (int c = 0; c < kCols; ++c)
        if (!((vis[(part * kCols + c) >> 5] >> (c & 31)) & 1u)) x[c] = -INFINITY;
    }
  };
  float top = -INFINITY;
#pragma unroll
  for (int part = 0; part < kParts; ++part) {
    load(part);
    float mx0 = x[0], mx1 = x[1], mx2 = x[2], mx3 = x[3];
#pragma unroll
    for (int c = 4; c + 8 <= kCols; c += 8) {
      mx0 = fmax3(mx0, x[c], x[c + 1]);
      mx1 = fmax3(mx1, x[c + 2], x[c + 3]);
      mx2 = fmax3(mx2, x[c + 4], x[c + 5]);
      mx3 = fmax3(mx3, x[c + 6], x[c + 7]);
    }
    mx0 = fmax3(mx0, x[kCols - 4], x[kCols - 3]);
    mx1 = fmax3(mx1, x[kCols - 2], x[kCols - 1]);
    top = fmaxf(top, fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)));
  }
  const float mx = fmaf(top, sl2, QUANT ? -kF16Lift : 0.f);
  const bool move = mx > m_run + kMaxSlack;
  const float m_new = move ? mx : m_run;
  const float m_new_use = (m_new == -INFINITY) ? 0.f : m_new;
  const float alpha = move ? ex2_approx(m_run - m_new_use) : 1.f;
  float sum0 = 0.f, sum1 = 0.f;
  // the last part first, which is here
#pragma unroll
  for (int part = kParts - 1; part >= 0; --part) {
    uint32_t pk[kCols / 32][16];
#pragma unroll
    for (int q = 0; q < kCols / 32; ++q) {
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        float a, b;
        ffma2(a, b, x[q * 32 + c], x[q * 32 + c + 1], sl2, sl2, -m_new_use, -m_new_use);
        a = ex2_approx(a);
        b = ex2_approx(b);
        fadd2(sum0, sum1, sum0, sum1, a, b);
        // P in 16 bits, the second product's operand type: off by at most 2^-8 (bf16) or
        // 2^-11 (f16) of each weight; l sums the unrounded values
        pk[q][c >> 1] = QUANT ? pack_f16x2(a, b) : pack_bf16x2(a, b);
      }
      if (part == 0) tmem_st16(s_addr + q * 16, pk[q]);
    }
    if (part > 0) {
      load(part - 1);  // (P lies over its columns)
#pragma unroll
      for (int q = 0; q < kCols / 32; ++q) tmem_st16(s_addr + part * (kCols / 2) + q * 16, pk[q]);
    }
  }
  l_run = l_run * alpha + (sum0 + sum1);
  rescale_row<D>(o_addr, has_o && (move || o_scale != 1.f), alpha * o_scale);
  tmem_wait_st();
  m_run = m_new;
  m_use = m_new_use;
}

// The same for a tile of codes with new keys, which enter the products as they are.  A key's scale
// must reach no row that does not see it, as one factor for a tile would: K's multiplies the score and
// V's the weight, relative to 2^ev of the row's, a power of two above all V scales that the row has
// seen (or, before, the exponent of the cached tiles).  ks, vs: the tile's scales in shared memory; good: the
// keys that the row sees and whose values are finite.
template <int D>
__device__ __forceinline__ void softmax_row_scaled(uint32_t s_addr, uint32_t o_addr, const uint32_t (&vis)[4],
                                                   const uint32_t (&good)[4], const float4* ks, const float4* vs,
                                                   bool has_o, float factor, int& ev, float& m_run, float& m_use,
                                                   float& l_run) {
  // (Loops over 32 keys at a time, since this code is met once or twice a piece: unrolled it takes
  // longer to fetch than to run, e4m3 trees of 26 at d = 64 48 us.)
  constexpr int kParts = BN / 32;
  uint32_t see[kParts], use[kParts];
#pragma unroll
  for (int i = 0; i < kParts; ++i) {
    see[i] = vis[i];
    use[i] = good[i];
  }
  auto turn = [](uint32_t (&w)[kParts]) {
    const uint32_t first = w[0];
#pragma unroll
    for (int i = 0; i + 1 < kParts; ++i) w[i] = w[i + 1];
    w[kParts - 1] = first;
  };
  float top = -INFINITY, most = 0.f;
#pragma unroll 1
  for (int part = 0; part < kParts; ++part) {
    uint32_t v[32];
    tmem_ld32(s_addr + part * 32, v);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < 32; c += 4) {
      const float4 k4 = ks[part * 8 + c / 4], v4 = vs[part * 8 + c / 4];
      const float k[4] = {k4.x, k4.y, k4.z, k4.w}, f[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = (see[0] >> (c + i)) & 1u ? __uint_as_float(v[c + i]) * score_factor(factor, k[i]) : -INFINITY;
        top = fmaxf(top, x);
        if ((use[0] >> (c + i)) & 1u) most = fmaxf(most, f[i]);
        v[c + i] = __float_as_uint(x);
      }
    }
    tmem_st32(s_addr + part * 32, v);
    turn(see);
    turn(use);
  }
  // (a factor is below 1, so that a weight of up to 2^15 stays one of f16)
  const int e = max(exponent_of(most) + 1, has_o ? ev : -126);
  const float o_scale = has_o ? exp2_int(max(ev - e, -126)) : 1.f, down = exp2_int(1 - e);
  ev = e;
  const float mx = top - kF16Lift;
  const bool move = mx > m_run + kMaxSlack;
  const float m_new = move ? mx : m_run;
  const float m_new_use = (m_new == -INFINITY) ? 0.f : m_new;
  const float alpha = move ? ex2_approx(m_run - m_new_use) : 1.f;
  float sum = 0.f;
  tmem_wait_st();
  // (P of a part lies over columns of S that have been loaded)
#pragma unroll 1
  for (int part = 0; part < kParts; ++part) {
    uint32_t v[32], pk[16];
    tmem_ld32(s_addr + part * 32, v);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < 32; c += 4) {
      const float4 v4 = vs[part * 8 + c / 4];
      const float f[4] = {v4.x, v4.y, v4.z, v4.w};
      float w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = ex2_approx(__uint_as_float(v[c + i]) - m_new_use);
        sum += w[i];
        w[i] = (use[0] >> (c + i)) & 1u ? w[i] * (f[i] * down * 0.5f) : 0.f;
      }
      // P in f16, off by at most 2^-11 of each weight; l sums the unrounded values
      pk[c / 2] = pack_f16x2(w[0], w[1]);
      pk[c / 2 + 1] = pack_f16x2(w[2], w[3]);
    }
    tmem_st16(s_addr + part * 16, pk);
    turn(use);
  }
  l_run = l_run * alpha + sum;
  rescale_row<D>(o_addr, has_o && (move || o_scale != 1.f), alpha * o_scale);
  tmem_wait_st();
  m_run = m_new;
  m_use = m_new_use;
}

// 16 columns from column 16 c on of row r of a piece: to the output, or to its partial.
__device__ __forceinline__ void put16(const TreeParams& p, const TreePiece& pc, int D, int r, int c, long long at,
                                      const float* f) {
  if (pc.slot >= 0) {
    float* dst = p.ws_o + (long long)pc.slot * p.unit_rows * D;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float x[8] = {f[8 * h], f[8 * h + 1], f[8 * h + 2], f[8 * h + 3],
                          f[8 * h + 4], f[8 * h + 5], f[8 * h + 6], f[8 * h + 7]};
      store8(dst + partial_at(2 * c + h, r, p.unit_rows), x);
    }
  } else if (p.o_f32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.o) + at * D + c * 16);
#pragma unroll
    for (int x = 0; x < 4; ++x) o[x] = make_float4(f[4 * x], f[4 * x + 1], f[4 * x + 2], f[4 * x + 3]);
  } else {
    uint32_t w[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) w[x] = pack_bf16x2(f[2 * x], f[2 * x + 1]);
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + at * D + c * 16;
    if (p.o_32)  // whole sectors
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                   "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                   : "memory");
    else {
      reinterpret_cast<uint4*>(o)[0] = make_uint4(w[0], w[1], w[2], w[3]);
      reinterpret_cast<uint4*>(o)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

template <int D, bool QUANT, bool DUAL>
__global__ void __launch_bounds__(MmaCfg<D, QUANT, DUAL>::kThreads, 1)
attn_tree_mma_kernel(const __grid_constant__ TreeMaps maps, const TreeParams p) {
  using C = MmaCfg<D, QUANT, DUAL>;
  constexpr int NS = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* empty = full + NS;
  uint64_t* raw_full = empty + NS;
  uint64_t* raw_empty = raw_full + C::kRawStages;
  uint64_t* q_full = raw_empty + C::kRawStages;
  uint64_t* q_empty = q_full + 2;
  uint64_t* s_full = q_empty + 2;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* bar_drain = o_full + 2;
  RawNote* raw_note = reinterpret_cast<RawNote*>(smem + C::kNoteOff);
  int2* tile_exp = reinterpret_cast<int2*>(smem + C::kExpOff);
  int8_t* q_lift = reinterpret_cast<int8_t*>(smem + C::kLiftOff);
  float* tail_scales = reinterpret_cast<float*>(smem + C::kTailOff);
  float2* ml = reinterpret_cast<float2*>(smem + C::kMlOff);
  int8_t* o_exp = reinterpret_cast<int8_t*>(smem + C::kEvOff);
  uint32_t* bad_scan = reinterpret_cast<uint32_t*>(smem + C::kBadOff);  // [2 streams][2][4]
  uint32_t* bad_slot = bad_scan + 16;                                   // [kStages][4] (e4m3)
  Pieces& pieces = *reinterpret_cast<Pieces*>(smem + C::kPiecesOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kWordOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* issued = reinterpret_cast<volatile int*>(tmem_slot + 2);  // K and V tiles, for the abort drain
  long long* found = reinterpret_cast<long long*>(tmem_slot + 4);
  auto& sums = *reinterpret_cast<long long (*)[C::kThreads / 32]>(smem + C::kSumOff);
  static_assert(C::kSumOff + sizeof(sums) <= C::kSmemBytes, "shared memory of the launch");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((smem_u32(smem) & 1023u) != 0) {  // the swizzled tiles need it (no static shared memory: it holds)
    if (threadIdx.x == 0) {
      set_status(p.status, CPATTN_ERR_ALIGNMENT);
      p.cut[2 * blockIdx.x + 1] = make_int4(0, 0, 0, 0);
    }
    return;
  }
  grid_dep_trigger();  // the merge may be scheduled as blocks of this grid end
  if (threadIdx.x == 0) {
    prefetch_tmap(&maps.k);
    prefetch_tmap(&maps.v);
    prefetch_tmap(&maps.k_tail);
    prefetch_tmap(&maps.v_tail);
    for (int i = 0; i < NS; ++i) {
      mbar_init(full + i, QUANT ? kConvertThreads : 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < C::kRawStages; ++i) {
      mbar_init(raw_full + i, 33);  // the TMA copies, with the note, and each lane's scales
      mbar_init(raw_empty + i, kConvertThreads);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(q_full + s, 1);
      mbar_init(q_empty + s, 1);
      mbar_init(s_full + s, 1);
      mbar_init(p_full + s, 128);
      mbar_init(o_full + s, 1);
    }
    mbar_init(bar_drain, 1);
    pieces.init(8);  // the softmax warps, whose end of a piece is the last
    *abort_flag = 0;
    issued[0] = issued[1] = 0;
    fence_barrier_init();
  }
  if (warp == kKWarp) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  const TreeStart start = tree_start(p, sums, found);  // (its barriers publish those above)
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t q_base = smem_u32(smem);
  const uint32_t ring_base = smem_u32(smem + C::kRingOff);

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsOther));
    if (warp == kKWarp || warp == kVWarp) {
      // ---------------------------------------------------------- producers --
      constexpr int kSt = QUANT ? C::kRawStages : NS;
      constexpr int kBytes = QUANT ? C::kRawTile : C::kTile;
      constexpr int kChunks = QUANT ? 1 : D / 64;   // boxes across a row
      constexpr int kLine = kBytes / BN / kChunks;  // bytes of a box row
      const bool is_v = warp == kVWarp;
      uint64_t* const fullb = QUANT ? raw_full : full;
      uint64_t* const emptyb = QUANT ? raw_empty : empty;
      uint8_t* const ring = smem + (QUANT ? C::kRawOff : C::kRingOff);
      const int whole_log = min(7, p.log_page);
      TileLoader<kPieces> w(pieces);
      int n = 0;
      bool ok = true;
      // (e4m3: a tile two ahead; bf16, where a tile takes longer: one)
      LoadTile cur = w.next(p, abort_flag), next{}, later{};
      if (QUANT) next = w.next(p, abort_flag);
      for (; cur.live; ++n) {
        if (QUANT) later = w.next(p, abort_flag);
        const int place = is_v ? v_place<!DUAL>(n) : k_place<!DUAL>(n), slot = place % kSt, row = cur.row(p);
        ok = wait_warp(emptyb + slot, ((place / kSt) & 1) ^ 1, abort_flag, p.timeout_ns);
        if (!ok) break;
        if (QUANT && lane == 0) raw_note[slot] = RawNote{cur.live, cur.fresh, cur.t <= (DUAL ? 0 : 1)};
        copy_tile<kChunks, kLine>(p, is_v ? &maps.v : &maps.k, is_v ? &maps.v_tail : &maps.k_tail,
                                  ring + slot * kBytes, fullb + slot, cur, row, whole_log);
        if constexpr (QUANT) {
          const uint32_t at = smem_u32(smem + C::kScaleOff + slot * BN * 8);
          copy_scales(p, is_v ? p.vs : p.ks, cur, row, at);
          if (!is_v) copy_scales(p, p.vs, cur, row, at + BN * 4);
          arrive_copies(fullb + slot);
        }
        cur = QUANT ? next : w.next(p, abort_flag);
        next = later;
      }
      if (QUANT) asm volatile("cp.async.wait_all;" ::: "memory");
      ok = ok && w.ok;
      if (lane == 0) {
        issued[is_v ? 1 : 0] = n;
        if (!ok) {
          set_status(p.status, CPATTN_ERR_TIMEOUT);
          *abort_flag = 1;
        }
      }
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------- MMA issuer --
      // The whole warp runs it and one lane issues: what the MMAs' descriptors are made of is
      // then uniform.  The pieces' tile counts come with their queries (0: no more).
      const uint32_t lead = lane == 0;
      constexpr uint32_t kIdescQK = idesc_16bit_f32(QUANT, BM, BN, 0);
      constexpr uint32_t kIdescPV = idesc_16bit_f32(QUANT, BM, D, 1);
      const uint64_t dq0 = smem_desc_sw128(q_base, 16, 1024);
      const uint64_t dk0 = smem_desc_sw128(ring_base, 16, 1024);
      const uint64_t dv0 = smem_desc_sw128(ring_base, BN * 128, 1024);
      auto issue_qk = [&](int s, int buf, int slot) {
        const uint64_t qd = dq0 + (uint32_t)(buf * (C::kQTile >> 4)), kd = dk0 + (uint32_t)(slot * (C::kTile >> 4));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          constexpr int kChunk = (BM * 128) >> 4;
          const uint64_t off = (uint64_t)((kk >> 2) * kChunk + (kk & 3) * 2);
          mma_ss_lead(lead, tmem_base + s * BN, qd + off, kd + off, kIdescQK, kk > 0 ? 1u : 0u);
        }
      };
      auto issue_pv = [&](int s, int slot, bool first) {
        const uint64_t vd = dv0 + (uint32_t)(slot * (C::kTile >> 4));
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)
          mma_ts_lead(lead, tmem_base + 2 * BN + s * D, tmem_base + s * BN + kk * 8,
                      vd + (uint64_t)(kk * ((16 * 128) >> 4)), kIdescPV, (!first || kk > 0) ? 1u : 0u);
      };
      auto commit = [&](uint64_t* bar) { mma_commit_lead(lead, bar); };
      auto wait = [&](uint64_t* bar, int parity) { return wait_warp(bar, parity, abort_flag, p.timeout_ns); };
      // P of a stream with the tile's V and, where it follows at once, the next K: every look at
      // a barrier is some 100 cycles in which the tensor core runs dry.
      auto wait_pv = [&](uint64_t* p_bar, int parity, uint64_t* v_bar, int v_parity, uint64_t* k_bar, int k_parity) {
        uint64_t t0 = 0;
        for (uint32_t i = 1;; ++i) {
          const bool x = mbar_try_wait(p_bar, parity), y = mbar_try_wait(v_bar, v_parity);
          const bool z = mbar_try_wait(k_bar, k_parity);
          if (__all_sync(0xffffffffu, x && y && z)) return true;
          if (i % kPollsPerCheck == 0 && __shfl_sync(0xffffffffu, (int)give_up(t0, abort_flag, p.timeout_ns), 0))
            return false;
        }
      };
      // Tiles of the pieces for the products Q K^T, which run ahead, and P V.
      int left_q = 0, left_v = 0;  // tiles of the piece behind the one at hand
      int piece_q = -1, piece_v = -1;
      uint32_t k_at = 0, v_at = DUAL ? 1 : 2;  // ring slots, and their phases
      uint32_t k_phase = 0, v_phase = 0;
      bool ok = true;
      bool head_v[2] = {false, false};
      auto advance = [&](uint32_t& slot, uint32_t& phase, uint32_t by) {
        slot += by;
        if (slot >= NS) {
          slot -= NS;
          phase ^= 1;
        }
      };
      // (the queries of a piece come after its place in the ring, which lasts until its end)
      auto tiles_of = [&](int i) { return __shfl_sync(0xffffffffu, pieces.at[i % kPieces].tiles, 0); };
      // The next tile's queries and K; false when there is none, or a wait ran out.
      auto next_q = [&]() {
        if (left_q == 0) {
          ++piece_q;
          const int buf = DUAL ? 0 : piece_q & 1;
          ok = wait(q_full + buf, (DUAL ? piece_q : piece_q >> 1) & 1);
          if (!ok) return false;
          left_q = tiles_of(piece_q);
          if (left_q == 0) return false;
          if (DUAL) ok = wait(q_full + 1, piece_q & 1);
        }
        --left_q;
        ok = ok && wait(full + k_at, k_phase);
        return ok;
      };
      // The next tile's V, its wait left to wait_pv (there is one wherever there was a next_q that
      // has not been followed).
      auto next_v = [&]() {
        if (left_v == 0) {
          ++piece_v;
          left_v = tiles_of(piece_v);
          head_v[0] = head_v[1] = true;
        }
        --left_v;
      };
      if constexpr (DUAL) {
        auto begin = [&](int s) {
          tc_fence_after();
          issue_qk(s, s, k_at);
          commit(s_full + s);
          if (left_q == 0) commit(q_empty + s);
        };
        auto begun = [&]() {
          commit(empty + k_at);
          advance(k_at, k_phase, 2);
        };
        bool more = next_q();
        if (more) {
          begin(0);
          begin(1);
          begun();
        }
        for (int n = 0; more && ok; ++n) {
          next_v();
          const bool last = left_v == 0;
          // (a next piece's queries may still be on their way: they do not hold up stream 1)
          const bool turn = left_q > 0;
          uint64_t* const v_bar = full + v_at;
          ok = wait_pv(p_full, n & 1, v_bar, v_phase, turn ? full + k_at : v_bar, turn ? k_phase : v_phase);
          if (!ok) break;
          tc_fence_after();
          issue_pv(0, v_at, head_v[0]);
          if (last) commit(o_full);
          if (turn) {
            --left_q;
            begin(0);
          }
          ok = wait(p_full + 1, n & 1);
          if (!ok) break;
          tc_fence_after();
          issue_pv(1, v_at, head_v[0]);
          head_v[0] = false;
          if (last) commit(o_full + 1);
          commit(empty + v_at);
          advance(v_at, v_phase, 2);
          if (!turn) {
            more = next_q();
            if (!more) break;
            begin(0);
          }
          begin(1);
          begun();
        }
      } else {
        int ahead = 0;  // tiles begun
        auto begin = [&](int s) {
          tc_fence_after();
          issue_qk(s, piece_q & 1, k_at);
          commit(s_full + s);
          commit(empty + k_at);
          if (left_q == 0) commit(q_empty + (piece_q & 1));
          advance(k_at, k_phase, ahead == 0 ? 1 : 2);
          ++ahead;
        };
        bool more = true;
        for (int s = 0; s < 2 && more; ++s) {
          more = next_q();
          if (more) begin(s);
        }
        for (int n = 0; n < ahead && ok; ++n) {
          const int s = n & 1;
          next_v();
          // (bf16 tiles come at the rate of HBM: a K on its way does not hold up the P V before it)
          const bool early = QUANT && left_q > 0;
          uint64_t* const v_bar = full + v_at;
          ok = wait_pv(p_full + s, (n >> 1) & 1, v_bar, v_phase, early ? full + k_at : v_bar, early ? k_phase : v_phase);
          if (!ok) break;
          tc_fence_after();
          issue_pv(s, v_at, head_v[s]);
          head_v[s] = false;
          if (left_v < 2) commit(o_full + s);
          commit(empty + v_at);
          advance(v_at, v_phase, 2);
          if (early) {
            --left_q;
            begin(s);
          } else if (more) {
            more = next_q();
            if (more) begin(s);
          }
        }
      }
      if (!ok && lane == 0) {
        set_status(p.status, CPATTN_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      // every MMA and commit issued by this thread has completed
      if (lane == 0) {
        mma_commit(bar_drain);
        wait_one(bar_drain, 0, nullptr, p.timeout_ns);
      }
    } else if (warp == kQWarp) {
      // -------------------------------------------------------------- queries --
      // D / 8 lanes to a row.  Dual: tile s of a piece in buffer s, when the piece before has
      // no product left; single: the pieces' tiles take turns, one ahead.
      constexpr int kLanes = D / 8, kRows = 32 / kLanes;
      // It also walks the share, two pieces ahead of the queries (of the first piece they are
      // on their way before the second is walked).
      TreeWalker<kPieces> walker(p, start, pieces);
      TreePiece pc;
      bool ok = true;
      const int c = lane % kLanes;
      int last[2] = {-1, -1};  // use of each buffer, where a box was its last
      for (int i = 0;; ++i) {
        walker.upto(p, i == 0 ? 0 : i + 2, abort_flag);
        ok = walker.ok && pieces.get(i, pc, abort_flag, p.timeout_ns);
        if (!ok) break;
        // (the end's queries are none, and published all the same: the MMA warp waits for them)
        const bool mine = !(QUANT && i == 0 && pc.tiles > 0);  // (else the softmax warps have them)
#pragma unroll
        for (int s = 0; s < (DUAL ? 2 : 1) && ok && mine; ++s) {
          const int buf = DUAL ? s : i & 1, use = DUAL ? i : i >> 1;
          ok = wait_warp(q_empty + buf, (use & 1) ^ 1, abort_flag, p.timeout_ns);
          if (!ok) break;
          const int rows = min(BM, pc.rows - s * BM);
          if (!QUANT && p.q_boxes) {  // a box holds all the heads of the tile's rows, packed as they are
            if (lane == 0 && !p.withhold_q) {
              if (rows > 0) {
                const int row = pc.row0 + group_div(p, pc.r0 + s * BM);
                mbar_arrive_expect_tx(q_full + buf, C::kQTile);
#pragma unroll
                for (int x = 0; x < D / 64; ++x)
                  tma_load_3d(smem + buf * C::kQTile + x * (BM * 128), &maps.q, q_full + buf, x * 64, pc.kv_head * p.g,
                              row);
                last[buf] = use;
              } else {
                mbar_arrive(q_full + buf);
                last[buf] = -1;  // (the box before has been used)
              }
            }
            continue;
          }
          const uint32_t tile = q_base + buf * C::kQTile + (c >> 3) * (BM * 128);
#pragma unroll 4
          for (int r = lane / kLanes; r < rows; r += kRows) {
            const int packed = pc.r0 + s * BM + r, node = group_div(p, packed);
            const __nv_bfloat16* src = p.q + (long long)(pc.row0 + node) * p.q_row +
                                       (long long)(pc.kv_head * p.g + packed - node * p.g) * p.q_head + c * 8;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tile + r * 128 + (((c & 7) ^ (r & 7)) << 4)),
                         "l"(src)
                         : "memory");
          }
        }
        if (!ok) break;
        if (i == 0) walker.upto(p, 2, abort_flag);
        if (pc.tiles) fetch_masks(p, pc);
        if (mine && (QUANT || !p.q_boxes)) {
          asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
          for (int s = 0; s < (DUAL ? 2 : 1); ++s) {
            const int buf = DUAL ? s : i & 1;
            if constexpr (QUANT) {
              // Each lane's own chunks, in place.  Loads of a batch before its stores: a chunk at a
              // time costs 230 cycles of latency.  (Rows of the batch behind the tile's last hold
              // anything.)
              constexpr int kBatch = 4;
              uint8_t* const tile = smem + buf * C::kQTile + (c >> 3) * (BM * 128);
              for (int r0 = lane / kLanes; r0 - lane / kLanes < pc.rows - s * BM && r0 < BM; r0 += kBatch * kRows) {
                uint4 x[kBatch];
                uint32_t mx[kBatch];
#pragma unroll
                for (int y = 0; y < kBatch; ++y) {
                  const int r = r0 + y * kRows;
                  x[y] = *reinterpret_cast<const uint4*>(tile + r * 128 + (((c & 7) ^ (r & 7)) << 4));
                  const uint32_t m = __vmaxu2(__vmaxu2(x[y].x & 0x7FFF7FFFu, x[y].y & 0x7FFF7FFFu),
                                              __vmaxu2(x[y].z & 0x7FFF7FFFu, x[y].w & 0x7FFF7FFFu));
                  mx[y] = max(m & 0xFFFFu, m >> 16);
                }
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
                  for (int y = 0; y < kBatch; ++y) mx[y] = max(mx[y], __shfl_xor_sync(0xffffffffu, mx[y], o));
#pragma unroll
                for (int y = 0; y < kBatch; ++y) {
                  const int r = r0 + y * kRows;
                  int f;
                  const QueryLift lift(mx[y], f);
                  *reinterpret_cast<uint4*>(tile + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = lift(x[y]);
                  if (c == 0) q_lift[i % C::kLifts * C::kLiftRows + s * BM + r] = (int8_t)f;
                }
              }
            }
            fence_async_shared();
            __syncwarp();
            if (lane == 0 && !p.withhold_q) mbar_arrive(q_full + buf);
          }
        }
        if (!pc.tiles) break;
      }
      if (lane == 0) {
        walker.end(p);
        if (!ok) {
          set_status(p.status, CPATTN_ERR_TIMEOUT);
          *abort_flag = 1;
        }
        // no copy in flight when the shared memory goes
        for (int buf = 0; buf < 2; ++buf)
          if (last[buf] >= 0) wait_one(q_full + buf, last[buf] & 1, nullptr, p.timeout_ns);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
    if constexpr (QUANT) if (warp >= kConvertWarp) {
      // --------------------------------------------------- codes to f16 tiles --
      // Warp w has rows 16w .. 16w+15 of every tile; of a row, lane l has 8 codes of each 64.
      constexpr int kMine = BN / kConvertWarps;  // rows of a warp
      const int w = warp - kConvertWarp;
      const int rl = lane >> 3, cl = lane & 7;  // row of four, 8-code chunk
      const uint32_t swz[2] = {(uint32_t)((cl ^ rl) << 4), (uint32_t)((cl ^ (rl + 4)) << 4)};
      constexpr int kBatch = 4, kHalves = D / 64;
      uint32_t from[2][kHalves];
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
          from[x][h] = code_at<D>(w * kMine + rl + 4 * x, h * 4 + (cl >> 1)) + (cl & 1) * 8;
      bool ok = true;
      // The KV tiles of the pieces so far; all: there are no more.
      int tiles = 0, piece = 0, ev_k[2] = {0, 0}, ev_v[2] = {0, 0};
      bool all = false;
      for (int place = 0; ok; ++place) {
        bool is_v;
        int n;
        if (DUAL) {
          is_v = place & 1;
          n = place >> 1;
        } else {
          is_v = place > 0 && !(place & 1);
          n = is_v ? (place - 2) >> 1 : (place + 1) >> 1;
        }
        while (!all && n >= tiles && ok) {
          TreePiece pc;
          ok = pieces.get(piece++, pc, abort_flag, p.timeout_ns);
          tiles += pc.tiles;
          all = pc.tiles == 0;
        }
        if (!ok || (n >= tiles && (is_v || DUAL))) break;
        if (n >= tiles) {  // (the place behind the last V but one)
          if (tiles == 0) break;
          continue;
        }
        const int raw = place % C::kRawStages, slot = place % NS;
        ok = wait_warp2(empty + slot, ((place / NS) & 1) ^ 1, raw_full + raw, (place / C::kRawStages) & 1, abort_flag,
                        p.timeout_ns);
        if (!ok) break;
        const RawNote note = raw_note[raw];
        const uint8_t* src = smem + C::kRawOff + raw * C::kRawTile;
        const float* scales = reinterpret_cast<const float*>(smem + C::kScaleOff + raw * BN * 8);
        // Exponents: K's factors are relative to the tile's largest scale, V's to the largest
        // that the stream has met in the piece (scales are not negative: their bits order as
        // integers).  Codes of a tile with new keys stay as they are (see softmax_row_scaled).
        const bool raw_codes = note.fresh < BN;
        float mx = 0.f, mv = 0.f;
        if (!raw_codes) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            mx = fmaxf(mx, scales[x * 32 + lane]);
            if (!is_v) mv = fmaxf(mv, scales[BN + x * 32 + lane]);
          }
        } else if (!is_v) {
          tail_scales[n % C::kTails * 2 * BN + w * 32 + lane] = scales[w * 32 + lane];
        }
        const int most = exponent_of(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx))));
        const int strm = DUAL ? 0 : n & 1;
        int e = most;
        // rows of this warp that become zeros
        uint32_t dead = note.live >= (w + 1) * kMine ? 0u : note.live <= w * kMine ? ~0u : ~0u << (note.live - w * kMine);
        if (!is_v) {
          const int v = exponent_of(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mv))));
          int& ev = strm ? ev_k[1] : ev_k[0];
          ev = note.first ? v : max(ev, v);
          if (w == 0 && lane == 0) tile_exp[n & 7] = make_int2(e, ev);
        } else {
          int& ev = strm ? ev_v[1] : ev_v[0];
          ev = note.first ? most : max(ev, most);
          e = ev;
          if (raw_codes) {  // new keys: a NaN's row
            const int row = w * kMine + lane / 2;  // two lanes to a row
            bool bad = !(scales[row] < INFINITY);
#pragma unroll
            for (int ch = 0; ch < D / 32; ++ch) {
              const uint4 v = *reinterpret_cast<const uint4*>(src + code_at<D>(row, (lane & 1) * (D / 32) + ch));
              bad = bad || __vcmpeq4(v.x & 0x7F7F7F7Fu, 0x7F7F7F7Fu) || __vcmpeq4(v.y & 0x7F7F7F7Fu, 0x7F7F7F7Fu) ||
                    __vcmpeq4(v.z & 0x7F7F7F7Fu, 0x7F7F7F7Fu) || __vcmpeq4(v.w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
            }
            const uint32_t word =
                __reduce_or_sync(0xffffffffu, bad && row >= note.fresh ? 1u << (lane / 2) : 0u) & ~dead;
            if (lane == 0) reinterpret_cast<uint16_t*>(bad_slot)[slot * kConvertWarps + w] = (uint16_t)word;
            dead |= word;
          }
        }
        const float inv = exp2_int(-e);
        dead >>= rl;
        const float* mul = scales + w * kMine + rl;
        uint8_t* dst = smem + C::kRingOff + slot * C::kTile + (w * kMine + rl) * 128;
        // loads of a batch before its stores: the compiler cannot tell them apart
#pragma unroll
        for (int r0 = 0; r0 < kMine; r0 += 4 * kBatch) {
          uint2 v[kBatch][kHalves];
          uint32_t m[kBatch];
#pragma unroll
          for (int x = 0; x < kBatch; ++x) {
            m[x] = pack_f16x2(raw_codes ? 1.f : mul[r0 + 4 * x] * inv, 0.f);
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
              v[x][h] = *reinterpret_cast<const uint2*>(src + from[x & 1][h] + (r0 + 4 * (x & ~1)) * D);
          }
          if (dead) {
#pragma unroll
            for (int x = 0; x < kBatch; ++x)
#pragma unroll
              for (int h = 0; h < kHalves; ++h)
                if ((dead >> (r0 + 4 * x)) & 1u) {
                  v[x][h] = make_uint2(0, 0);
                  m[x] = 0;
                }
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
        mbar_arrive(full + slot);
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
    // A wait that runs out leaves ok false for good: no more waits, but every barrier of the
    // warps still comes, so that none is left behind in one.
    const int s = warp >> 2;          // stream
    const int wq = warp & 3;          // TMEM lane quarter
    const int trow = wq * 32 + lane;  // row within the MMA tile
    const int r = DUAL ? s * BM + trow : trow;  // within the unit
    const uint32_t lanes = tmem_base + ((uint32_t)(wq * 32) << 16);
    const uint32_t s_addr = lanes + s * BN, o_addr = lanes + 2 * BN + s * D;
    TreePiece pc;
    bool ok = true, pending = false;  // pending: the other stream may still read this one's O
    int n0 = 0;                       // KV tiles before the piece
    int tails = 0;                    // of the stream, with new keys
    int had[2] = {0, 0};              // pieces in which a stream had tiles
    if constexpr (QUANT) {
      // The first piece's queries, a row a thread: one warp takes microseconds to bring 256 rows
      // and to turn them, in which these have nothing to do (trees of 26 at d = 64 35.1 -> 31.8
      // us, of 64 440 -> 431, of 32 306 -> 293).
      ok = pieces.get(0, pc, abort_flag, p.timeout_ns);
      if (DUAL || s == 0) {
        if (ok && r < pc.rows) {
          const int packed = pc.r0 + r, node = group_div(p, packed);
          const uint4* src = reinterpret_cast<const uint4*>(
              p.q + (long long)(pc.row0 + node) * p.q_row + (long long)(pc.kv_head * p.g + packed - node * p.g) * p.q_head);
          uint4 v[D / 8];
#pragma unroll
          for (int c = 0; c < D / 8; ++c) v[c] = __ldg(src + c);
          uint32_t mx = 0;
#pragma unroll
          for (int c = 0; c < D / 8; ++c)
            mx = __vmaxu2(__vmaxu2(mx, __vmaxu2(v[c].x & 0x7FFF7FFFu, v[c].y & 0x7FFF7FFFu)),
                          __vmaxu2(v[c].z & 0x7FFF7FFFu, v[c].w & 0x7FFF7FFFu));
          int f;
          const QueryLift lift(max(mx & 0xFFFFu, mx >> 16), f);
          uint8_t* const line = smem + s * C::kQTile + trow * 128;
#pragma unroll
          for (int c = 0; c < D / 8; ++c)
            *reinterpret_cast<uint4*>(line + (c >> 3) * (BM * 128) + (((c & 7) ^ (trow & 7)) << 4)) = lift(v[c]);
          q_lift[s * BM + trow] = (int8_t)f;
        }
        fence_async_shared();
        bar_named(2 + s, 128);
        if (trow == 0 && ok && pc.tiles > 0 && !p.withhold_q) mbar_arrive(q_full + s);
      }
    }
    for (int i = 0;; ++i) {
      ok = ok && pieces.get(i, pc, abort_flag, p.timeout_ns);
      if (!bar_all(6, ok && pc.tiles > 0)) break;  // (all eight warps go on, or none)
      const bool warp_live = (r & ~31) < pc.rows;
      const int node = r < pc.rows ? group_div(p, pc.r0 + r) : 0;
      float m_run = -INFINITY, l_run = 0.f, m_use = 0.f, factor = p.scale_log2;
      int ev = 0;  // exponent of O
      bool first = true;
      for (int t = DUAL ? 0 : (n0 ^ s) & 1; t < pc.tiles; t += DUAL ? 1 : 2) {
        const int n = n0 + t, key0 = (pc.t0 + t) * BN;
        // tiles with new keys, or keys behind the last
        const bool tail = key0 + BN > pc.L;
        MaskWords words;
        if (tail && warp_live) words.load(p, pc, node, key0 - pc.L);
        ok = ok && wait_warp(s_full + s, (DUAL ? n : n >> 1) & 1, abort_flag, p.timeout_ns);
        tc_fence_after();
        float sl2 = factor, o_scale = 1.f;
        if constexpr (QUANT) {
          if (first && r < pc.rows) factor = p.scale_log2 * exp2_int(-q_lift[i % C::kLifts * C::kLiftRows + r]);
          // written before the K tile went to the tensor core, and not again before this
          // step's P has been used
          if (!tail) {
            const volatile int2* e = tile_exp + (n & 7);
            const int ek = e->x, ev_now = e->y;
            sl2 = score_factor(factor, exp2_int(ek));
            if (!first && ev_now != ev) o_scale = exp2_int(max(ev - ev_now, -126));
            ev = ev_now;
          }
        }
        uint32_t vis[4] = {~0u, ~0u, ~0u, ~0u}, good[4] = {0, 0, 0, 0};
        float poison = 0.f;
        if (tail) {
          const int slot = v_place<!DUAL>(n) % NS;
          if (warp_live) words.seen(key0 - pc.L, p.mask ? pc.T : node + 1, vis);
          ok = ok && wait_warp(full + slot, (v_place<!DUAL>(n) / NS) & 1, abort_flag, p.timeout_ns);
          const uint32_t* bad_words;
          if constexpr (!QUANT) {
            // value row trow of the tile: one of no key, or one that is not finite
            uint8_t* const line = smem + C::kRingOff + slot * C::kTile + trow * 128;
            auto chunk_at = [&](int c) { return (c >> 3) * (BN * 128) + ((c ^ trow) & 7) * 16; };
            const int key = key0 + trow;
            bool bad = false;
            if (key >= pc.L && key < pc.keys) {
#pragma unroll
              for (int c = 0; c < D / 8; ++c) {
                const uint4 v = *reinterpret_cast<const uint4*>(line + chunk_at(c));
                bad = bad || __vcmpgeu2(v.x & 0x7FFF7FFFu, 0x7F807F80u) || __vcmpgeu2(v.y & 0x7FFF7FFFu, 0x7F807F80u) ||
                      __vcmpgeu2(v.z & 0x7FFF7FFFu, 0x7F807F80u) || __vcmpgeu2(v.w & 0x7FFF7FFFu, 0x7F807F80u);
              }
            }
            uint32_t* const mine = bad_scan + (s * 2 + (tails & 1)) * 4;
            const uint32_t word = __ballot_sync(0xffffffffu, bad);
            if (lane == 0) mine[wq] = word;
            bad_words = mine;
            ++tails;
            if (DUAL) bar_named(2, 256);  // both streams have looked at the tile
            else bar_named(2 + s, 128);
            if (bad || key >= pc.keys) {
#pragma unroll
              for (int c = 0; c < D / 8; ++c)
                *reinterpret_cast<uint4*>(line + chunk_at(c)) = make_uint4(0, 0, 0, 0);
            }
            fence_async_shared();
          } else {
            bad_words = bad_slot + slot * 4;
          }
          uint32_t hit = 0;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            hit |= vis[x] & bad_words[x];
            if (QUANT) good[x] = vis[x] & ~bad_words[x];
          }
          if (r < pc.rows && hit) poison = __uint_as_float(0x7FC00000u);
        }
        if (warp_live && ok) {
          if (QUANT && tail) {
            const float4* const ks = reinterpret_cast<const float4*>(tail_scales + n % max(C::kTails, 1) * 2 * BN);
            softmax_row_scaled<D>(s_addr, o_addr, vis, good, ks, ks + BN / 4, !first, factor, ev, m_run, m_use, l_run);
          } else {
            softmax_row<D, QUANT>(s_addr, o_addr, tail, vis, !first, o_scale, sl2, m_run, m_use, l_run);
          }
        }
        l_run += poison;
        first = false;
        if (!DUAL && pending) {
          bar_named(5, 256);
          pending = false;
        }
        tc_fence_before();
        mbar_arrive(p_full + s);
      }
      // ---- the piece's end ----
      const int packed = pc.r0 + r;
      const long long at = (long long)(pc.row0 + node) * p.Hq + pc.kv_head * p.g + packed - node * p.g;
      if constexpr (DUAL) {
        ok = ok && wait_warp(o_full + s, i & 1, abort_flag, p.timeout_ns);
        tc_fence_after();
        if (warp_live && ok) {
          const bool none = l_run == 0.f;  // (a NaN sum is not none)
          const float inv = none ? 0.f : exp2_int(ev) / l_run;
#pragma unroll
          for (int q = 0; q < D / 64; ++q) {
            uint32_t v[64];
            tmem_ld32p(o_addr + q * 64, v);
            tmem_ld32p(o_addr + q * 64 + 32, v + 32);
            tmem_wait_ld();
            if (r < pc.rows) {
#pragma unroll
              for (int c = 0; c < 64; c += 16) {
                float f[16];
#pragma unroll
                for (int x = 0; x < 16; ++x) f[x] = none ? 0.f : __uint_as_float(v[c + x]) * inv;
                put16(p, pc, D, r, q * 4 + c / 16, at, f);
              }
            }
          }
          if (r < pc.rows) {
            const float lse2 = none ? -INFINITY : m_use + lg2_approx(l_run);
            if (pc.slot >= 0) p.ws_l[(long long)pc.slot * p.unit_rows + r] = lse2;
            else p.lse[at] = lse2 * kLn2;
          }
        }
        tc_fence_before();
      } else {
        if (pending) bar_named(5, 256);
        ml[s * BM + trow] = make_float2(m_use, l_run);
        if constexpr (QUANT) o_exp[s * BM + trow] = (int8_t)ev;
        bar_named(4, 256);
        // the streams that had tiles (an O of none is not looked at)
        bool live[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          live[x] = pc.tiles > 1 || (n0 & 1) == x;
          if (live[x]) ok = ok && wait_warp(o_full + x, had[x]++ & 1, abort_flag, p.timeout_ns);
        }
        tc_fence_after();
        if (warp_live && ok) {
          const float2 a = ml[trow], b = ml[BM + trow];
          const float ua = QUANT ? exp2_int(o_exp[trow]) : 1.f, ub = QUANT ? exp2_int(o_exp[BM + trow]) : 1.f;
          // (m of a stream without keys means nothing)
          float M = fmaxf(a.y != 0.f ? a.x : -INFINITY, b.y != 0.f ? b.x : -INFINITY);
          if (M == -INFINITY) M = 0.f;
          const float fa = a.y != 0.f ? ex2_approx(a.x - M) : 0.f, fb = b.y != 0.f ? ex2_approx(b.x - M) : 0.f;
          const float sum = (a.y != 0.f ? fa * a.y : 0.f) + (b.y != 0.f ? fb * b.y : 0.f);
          const bool none = sum == 0.f;
          const float inv = none ? 0.f : 1.f / sum;
          const float ca = live[0] ? fa * inv * ua : 0.f, cb = live[1] ? fb * inv * ub : 0.f;
          const uint32_t from = lanes + 2 * BN + s * (D / 2);  // this stream's half of the columns
#pragma unroll
          for (int q = 0; q < D / 64; ++q) {
            uint32_t u[32], v[32];
            tmem_ld32(from + q * 32, u);
            tmem_ld32(from + D + q * 32, v);
            tmem_wait_ld();
            if (r < pc.rows) {
#pragma unroll
              for (int c = 0; c < 32; c += 16) {
                float f[16];
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                  const float y = ca == 0.f ? 0.f : __uint_as_float(u[c + x]) * ca;
                  f[x] = cb == 0.f ? y : fmaf(__uint_as_float(v[c + x]), cb, y);
                }
                put16(p, pc, D, r, s * (D / 32) + q * 2 + c / 16, at, f);
              }
            }
          }
          if (r < pc.rows && s == 0) {
            const float lse2 = none ? -INFINITY : M + lg2_approx(sum);
            if (pc.slot >= 0) p.ws_l[(long long)pc.slot * p.unit_rows + r] = lse2;
            else p.lse[at] = lse2 * kLn2;
          }
        }
        tc_fence_before();
        pending = true;
      }
      n0 += pc.tiles;
      __syncwarp();
      if (lane == 0) pieces.done(i);
    }
    if (!ok && lane == 0) {
      set_status(p.status, CPATTN_ERR_TIMEOUT);
      *abort_flag = 1;
    }
  }

  // ---- teardown ----
  tc_fence_before();
  __syncthreads();
  if (warp == kKWarp) {
    // (after an abort) let the copies in flight land before the shared memory goes
    if (lane == 0 && *abort_flag)
      drain_tiles<!DUAL>(QUANT ? raw_full : full, QUANT ? C::kRawStages : NS, issued[0], issued[1], p.timeout_ns);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

template <int D, bool QUANT, bool DUAL>
int launch(const TreeMaps& m, const TreeParams& p, int num_ctas, cudaStream_t stream) {
  using C = MmaCfg<D, QUANT, DUAL>;
  auto kern = attn_tree_mma_kernel<D, QUANT, DUAL>;
  if (!allow_smem(kern, C::kSmemBytes)) return CPATTN_ERR_CUDA;
  static std::atomic<int> covered{0};
  if (!split_covered(kern, C::kThreads, C::kRegsSoftmax * 256 + C::kRegsOther * (C::kThreads - 256), covered)) return CPATTN_ERR_UNSUPPORTED;
  return launch_kernel(kern, (unsigned)num_ctas, C::kThreads, C::kSmemBytes, stream, false, m, p) == cudaSuccess
             ? CPATTN_OK
             : CPATTN_ERR_CUDA;
}
template <bool DUAL>
int launch(const TreeMaps& m, const TreeParams& p, int d, bool quant, int num_ctas, cudaStream_t stream) {
  return d == 128 ? (quant ? launch<128, true, DUAL>(m, p, num_ctas, stream)
                           : launch<128, false, DUAL>(m, p, num_ctas, stream))
                  : (quant ? launch<64, true, DUAL>(m, p, num_ctas, stream)
                           : launch<64, false, DUAL>(m, p, num_ctas, stream));
}

}  // namespace

int launch_tree_mma(const TreeMaps& m, const TreeParams& p, int d, bool quant, int num_ctas, cudaStream_t stream) {
  return p.unit_rows == BM ? launch<false>(m, p, d, quant, num_ctas, stream)
                           : launch<true>(m, p, d, quant, num_ctas, stream);
}

}  // namespace cpattn
