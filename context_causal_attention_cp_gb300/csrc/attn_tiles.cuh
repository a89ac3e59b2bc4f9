// Pieces of the attention kernels over cached rows (attn_shared.cu, attn_tree.cu): bounded
// waits, tiles of codes, 16-bit arithmetic, warp-level MMAs and partial rows.
#pragma once
#include <cstdint>

#include "attn_common.cuh"
#include "shared_plan.h"

namespace cpattn {
namespace {

constexpr int BN = kSharedTileKeys;  // keys of a KV tile

// Orders this thread's shared-memory accesses before later ones of the async proxy (TMA,
// tcgen05.mma reading shared memory).
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

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
template <class Params>
__device__ __forceinline__ int group_div(const Params& p, int n) {
  return p.g == 1 ? n : (int)(__umulhi((uint32_t)n, p.g_mul) >> p.g_shift);
}

__device__ __forceinline__ int num_tiles(int keys) { return (keys - 1) / BN + 1; }

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

template <bool F16>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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
__device__ __forceinline__ float lds_f32(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t c) {  // the low half
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  return h;
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {  // 16-bit elements
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// 3-D map of a code buffer (cols, heads, rows) with a D-column x 1-head box, rows
// packed in shared memory and swizzled over their length (see code_at); out-of-range
// rows read as zero.
inline bool make_code_map(CUtensorMap* m, const void* base, int cols, int heads, long long rows,
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

}  // namespace
}  // namespace cpattn
