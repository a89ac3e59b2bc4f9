// Quantised KV cache: write (bf16 / fp32 rows to e4m3 codes with a power-of-two
// scale per row and head) and read back.
//
// For one vector x: a = max finite |x_c|, e = clamp(ceil(log2(a/448)), -117,
// 119), scale = 2^e, code_c = e4m3(x_c 2^-e), value = code_c 2^e.  Both kernels
// are HBM streams: a vector is read once, kept in registers between the maximum
// and the rounding, and its codes are written once.  L = 2^k lanes share a vector,
// 8 elements each and step, so that a load or store of a step has no gaps (16 elements
// left every store two passes over its lines: 32768 rows of 16 vectors of 128 read back
// in 45 us; now 36).  L is the smallest that leaves a lane at most four steps: with L twice or four
// times that, the shuffles of the maximum and the walk over rows cost more (8192 rows
// of 16 vectors of 128: 12 us, 15 and 21).  A thread works on kUnroll rows at once, so
// that their loads travel together (one row where a lane has three steps or more: 16384
// rows of 576 take 10 us, as long as 1.7 times their bytes in rows of 128); which row,
// side and head it has is settled once, before its loop over rows.
#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>

#include "../../include/cpattn.h"
#include "kv_codes.cuh"
#include "ptx.cuh"
#include "trace.h"

namespace cpattn {
namespace {

constexpr int kKvThreads = 256;
constexpr int kWriteBlocks = 4, kReadBlocks = 5;  // resident on an SM
constexpr int kMaxDim = 1024;

struct KvSide {  // one of K and V
  const void* x;
  long long x_row, x_head;  // elements
  uint8_t* codes;
  float* scales;
  long long c_row, c_head, s_head;
  void* out;
  int dim;
};

constexpr int kChunk = 8;  // elements of a lane's step: 16 bytes of bf16, 8 of codes

// 8 consecutive elements, as they lie in memory.
template <bool F32>
struct Raw8 {
  static constexpr int kWords = F32 ? 2 : 1;
  uint4 w[kWords];
  __device__ __forceinline__ void load(const void* x, long long at) {
    const uint4* p = F32 ? reinterpret_cast<const uint4*>(static_cast<const float*>(x) + at)
                         : reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at);
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __ldcs(p + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ float at(int c) const {  // c a constant
    const uint4& v = w[c / (F32 ? 4 : 8)];
    const int i = F32 ? c % 4 : c % 8 / 2;
    const uint32_t u = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    return __uint_as_float(F32 ? u : c % 2 ? u & 0xFFFF0000u : u << 16);
  }
  // max |x_c| with the bits of an infinity or NaN above all numbers'
  __device__ __forceinline__ uint32_t max_bits() const {
    if constexpr (F32) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        m = max(max(m, max(w[i].x & 0x7FFFFFFFu, w[i].y & 0x7FFFFFFFu)),
                max(w[i].z & 0x7FFFFFFFu, w[i].w & 0x7FFFFFFFu));
      return m;
    } else {
      const uint32_t m = __vmaxu2(__vmaxu2(w[0].x & 0x7FFF7FFFu, w[0].y & 0x7FFF7FFFu),
                                  __vmaxu2(w[0].z & 0x7FFF7FFFu, w[0].w & 0x7FFF7FFFu));
      return max(m & 0xFFFF0000u, m << 16);
    }
  }
  __device__ __forceinline__ float max_finite() const {
    float a = 0.f;
#pragma unroll
    for (int c = 0; c < kChunk; ++c) {
      const float m = fabsf(at(c));
      a = fmaxf(a, m < INFINITY ? m : 0.f);
    }
    return a;
  }
};

// A thread's place: row `row` of the block's rows, vector (side, head) and lane.  A
// block has kKvThreads / (vectors * L) rows, or one row in several passes.
struct KvPlace {
  int row, rows, first;  // first: its (vector, lane) number, the others follow by kKvThreads
  bool on;
};
__device__ __forceinline__ KvPlace kv_place(int lanes_per_row) {
  KvPlace p;
  p.rows = max(1, kKvThreads / lanes_per_row);
  p.row = (int)threadIdx.x / lanes_per_row;
  p.on = p.row < p.rows || lanes_per_row > kKvThreads;
  if (lanes_per_row > kKvThreads) p.row = 0;
  p.first = (int)threadIdx.x - p.row * lanes_per_row;
  return p;
}

// NC: chunks of a lane (dim <= 8 * L * NC).
template <bool F32, int NC>
__global__ void __launch_bounds__(kKvThreads)
kv_quantize_kernel(const KvSide k, const KvSide v, int sides, int num_rows, int Hkv, int log_l,
                   const int32_t* __restrict__ slots, int cache_rows, int32_t* status) {
  constexpr int kUnroll = F32 ? (NC == 1 ? 2 : 1) : NC == 1 ? 4 : NC == 2 ? 2 : 1;
  const int L = 1 << log_l, lpr = (sides * Hkv) << log_l;
  const KvPlace pl = kv_place(lpr);
  if (!pl.on) return;
  const uint32_t group = (L == 32 ? 0xffffffffu : (1u << L) - 1u) << (threadIdx.x & 31 & ~(L - 1));
  const int step = gridDim.x * pl.rows;
  for (int x = pl.first; x < lpr; x += kKvThreads) {
    const int vec = x >> log_l, lane = x & (L - 1);
    const KvSide& s = vec >= Hkv ? v : k;
    const int h = vec >= Hkv ? vec - Hkv : vec;
    const int c0 = lane * kChunk;
    for (long long r0 = (long long)blockIdx.x * pl.rows + pl.row; r0 < num_rows;
         r0 += (long long)step * kUnroll) {
      Raw8<F32> raw[kUnroll][NC];
      int slot[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const long long row = r0 + (long long)u * step;
        slot[u] = row < num_rows ? (slots ? __ldg(slots + row) : (int)row) : -1;
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const long long row = r0 + (long long)u * step;
        if (slot[u] >= cache_rows) {
          if (lane == 0) set_status(status, CPATTN_ERR_RANGE);
          slot[u] = -1;
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int c = c0 + i * L * kChunk;
          if (slot[u] >= 0 && c < s.dim) raw[u][i].load(s.x, row * s.x_row + h * s.x_head + c);
          else raw[u][i].zero();
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        uint32_t bits = 0;
#pragma unroll
        for (int i = 0; i < NC; ++i) bits = max(bits, raw[u][i].max_bits());
        for (int o = L >> 1; o > 0; o >>= 1) bits = max(bits, __shfl_xor_sync(group, bits, o));
        float a = __uint_as_float(bits);
        if (bits >= 0x7F800000u) {  // (the same in the vector's lanes)
          a = 0.f;
#pragma unroll
          for (int i = 0; i < NC; ++i) a = fmaxf(a, raw[u][i].max_finite());
          for (int o = L >> 1; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(group, a, o));
        }
        if (slot[u] < 0) continue;
        const int e = scale_exponent(a);
        const float inv = exp2_int(-e);
        uint8_t* dst = s.codes + (long long)slot[u] * s.c_row + h * s.c_head;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int c = c0 + i * L * kChunk;
          if (c >= s.dim) continue;
          uint32_t w[2];
#pragma unroll
          for (int j = 0; j < 2; ++j)
            w[j] = (uint32_t)e4m3x2(raw[u][i].at(4 * j) * inv, raw[u][i].at(4 * j + 1) * inv) |
                   (uint32_t)e4m3x2(raw[u][i].at(4 * j + 2) * inv, raw[u][i].at(4 * j + 3) * inv) << 16;
          *reinterpret_cast<uint2*>(dst + c) = make_uint2(w[0], w[1]);
        }
        if (lane == 0) s.scales[h * s.s_head + slot[u]] = exp2_int(e);
      }
    }
  }
}

template <bool F32, int NC>
__global__ void __launch_bounds__(kKvThreads, kReadBlocks)
kv_dequantize_kernel(const KvSide k, const KvSide v, int sides, int num_rows, int Hkv, int log_l,
                     const int32_t* __restrict__ idx, int cache_rows, int32_t* status) {
  constexpr int kUnroll = NC == 1 ? 4 : NC == 2 ? 2 : 1;
  const int L = 1 << log_l, lpr = (sides * Hkv) << log_l;
  const KvPlace pl = kv_place(lpr);
  if (!pl.on) return;
  const int step = gridDim.x * pl.rows;
  for (int x = pl.first; x < lpr; x += kKvThreads) {
    const int vec = x >> log_l, lane = x & (L - 1);
    const KvSide& s = vec >= Hkv ? v : k;
    const int h = vec >= Hkv ? vec - Hkv : vec;
    const int c0 = lane * kChunk;
    for (long long r0 = (long long)blockIdx.x * pl.rows + pl.row; r0 < num_rows;
         r0 += (long long)step * kUnroll) {
      int src[kUnroll];
      float scale[kUnroll];
      uint2 w[kUnroll][NC];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const long long row = r0 + (long long)u * step;
        src[u] = row < num_rows ? (idx ? __ldg(idx + row) : (int)row) : -1;
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (src[u] >= cache_rows) {
          if (lane == 0) set_status(status, CPATTN_ERR_RANGE);
          src[u] = -1;
        }
        if (src[u] < 0) continue;
        scale[u] = __ldg(s.scales + h * s.s_head + src[u]);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int c = c0 + i * L * kChunk;
          if (c < s.dim)
            w[u][i] = __ldg(reinterpret_cast<const uint2*>(s.codes + (long long)src[u] * s.c_row +
                                                           h * s.c_head + c));
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (src[u] < 0) continue;
        const long long at = ((r0 + (long long)u * step) * Hkv + h) * s.dim;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int c = c0 + i * L * kChunk;
          if (c >= s.dim) continue;
          const uint32_t q[2] = {w[u][i].x, w[u][i].y};
          float f[kChunk];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            e4m3x2_to_f32((uint16_t)q[j], f[4 * j], f[4 * j + 1]);
            e4m3x2_to_f32((uint16_t)(q[j] >> 16), f[4 * j + 2], f[4 * j + 3]);
          }
#pragma unroll
          for (int j = 0; j < kChunk; ++j) f[j] *= scale[u];
          if (F32) {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(s.out) + at + c);
#pragma unroll
            for (int j = 0; j < 2; ++j)
              __stcs(o + j, make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]));
          } else {
            __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(s.out) + at + c),
                   make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                              pack_bf16x2(f[6], f[7])));
          }
        }
      }
    }
  }
}

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Checks one side's cache and moves it into the kernels' form.
int cache_side(const cp_kv_codes_t* c, int dim, int Hkv, int cache_rows, KvSide* s) {
  if (dim < 16 || dim > kMaxDim || dim % 16) return CPATTN_ERR_UNSUPPORTED;
  if ((!c->codes || !c->scales) && cache_rows > 0) return CPATTN_ERR_INVALID_ARG;
  if (!aligned(c->codes, 16) || !aligned(c->scales, 4) || c->row_stride % 16 ||
      c->head_stride % 16)
    return CPATTN_ERR_ALIGNMENT;
  if (c->head_stride < dim || c->row_stride < (int64_t)(Hkv - 1) * c->head_stride + dim ||
      c->scale_stride < cache_rows)
    return CPATTN_ERR_INVALID_ARG;
  s->codes = static_cast<uint8_t*>(c->codes);
  s->scales = c->scales;
  s->c_row = c->row_stride;
  s->c_head = c->head_stride;
  s->s_head = c->scale_stride;
  s->dim = dim;
  return CPATTN_OK;
}

// Lanes of a vector (log2) and blocks of a launch: enough for the rows, and at most as
// many as reside at once, the rest of the rows being the loop's (16 per SM, in turn:
// 8192 rows written in 14 us instead of 12).  Reading, five blocks that hold half as many
// rows each in flight beat four (36.5 and 38 us for 32768 rows).
struct KvShape {
  int log_l, chunks;
  unsigned grid;
};
KvShape kv_shape(int num_rows, int vectors, int dim, int blocks_per_sm) {
  KvShape s;
  for (s.log_l = 0; s.log_l < 5 && (4 * kChunk << s.log_l) < dim; ++s.log_l) {}
  s.chunks = (dim + (kChunk << s.log_l) - 1) / (kChunk << s.log_l);
  const long long lpr = (long long)vectors << s.log_l, rows = std::max<long long>(1, kKvThreads / lpr);
  s.grid = (unsigned)std::min<long long>((num_rows + rows - 1) / rows, 152 * blocks_per_sm);
  return s;
}

}  // namespace
}  // namespace cpattn

using namespace cpattn;

extern "C" int cp_kv_quantize(const void* k, int64_t k_row_stride, int64_t k_head_stride,
                              const void* v, int64_t v_row_stride, int64_t v_head_stride,
                              int x_is_fp32, int num_rows, int Hkv, int d, int dv,
                              const int32_t* slots, const cp_kv_codes_t* k_cache,
                              const cp_kv_codes_t* v_cache, int cache_rows, int32_t* status_dev,
                              cudaStream_t stream) {
  CPATTN_TRACE("cp_kv_quantize");
  if (num_rows < 0 || cache_rows < 0 || Hkv < 1 || !k_cache) return CPATTN_ERR_INVALID_ARG;
  KvSide ks{}, vs{};
  int rc = cache_side(k_cache, d, Hkv, cache_rows, &ks);
  if (rc == CPATTN_OK && v_cache) rc = cache_side(v_cache, dv, Hkv, cache_rows, &vs);
  if (rc != CPATTN_OK) return rc;
  const int64_t per16 = x_is_fp32 ? 4 : 8;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4) || k_row_stride % per16 ||
      k_head_stride % per16 || (v && (v_row_stride % per16 || v_head_stride % per16)))
    return CPATTN_ERR_ALIGNMENT;
  if (k_row_stride < 0 || k_head_stride < 0 || (v && (v_row_stride < 0 || v_head_stride < 0)))
    return CPATTN_ERR_INVALID_ARG;
  if (num_rows == 0) return CPATTN_OK;
  if (!k || (v != nullptr) != (v_cache != nullptr)) return CPATTN_ERR_INVALID_ARG;
  ks.x = k;
  ks.x_row = k_row_stride;
  ks.x_head = k_head_stride;
  vs.x = v;
  vs.x_row = v_row_stride;
  vs.x_head = v_head_stride;
  const int sides = v ? 2 : 1;
  const KvShape sh = kv_shape(num_rows, sides * Hkv, std::max(d, v ? dv : 0), kWriteBlocks);
  decltype(&kv_quantize_kernel<true, 1>) const kerns[2][4] = {
      {kv_quantize_kernel<false, 1>, kv_quantize_kernel<false, 2>, kv_quantize_kernel<false, 3>,
       kv_quantize_kernel<false, 4>},
      {kv_quantize_kernel<true, 1>, kv_quantize_kernel<true, 2>, kv_quantize_kernel<true, 3>,
       kv_quantize_kernel<true, 4>}};
  auto kern = kerns[x_is_fp32 ? 1 : 0][sh.chunks - 1];
  kern<<<sh.grid, kKvThreads, 0, stream>>>(ks, vs, sides, num_rows, Hkv, sh.log_l, slots, cache_rows,
                                           status_dev);
  return cudaGetLastError() == cudaSuccess ? CPATTN_OK : CPATTN_ERR_CUDA;
}

extern "C" int cp_kv_dequantize(const cp_kv_codes_t* k_cache, const cp_kv_codes_t* v_cache,
                                int cache_rows, int Hkv, int d, int dv, const int32_t* idx,
                                int num_rows, void* k_out, void* v_out, int out_is_fp32,
                                int32_t* status_dev, cudaStream_t stream) {
  CPATTN_TRACE("cp_kv_dequantize");
  if (num_rows < 0 || cache_rows < 0 || Hkv < 1 || !k_cache) return CPATTN_ERR_INVALID_ARG;
  KvSide ks{}, vs{};
  int rc = cache_side(k_cache, d, Hkv, cache_rows, &ks);
  if (rc == CPATTN_OK && v_cache) rc = cache_side(v_cache, dv, Hkv, cache_rows, &vs);
  if (rc != CPATTN_OK) return rc;
  if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(idx, 4)) return CPATTN_ERR_ALIGNMENT;
  if (num_rows == 0) return CPATTN_OK;
  if (!k_out || (v_out != nullptr) != (v_cache != nullptr)) return CPATTN_ERR_INVALID_ARG;
  ks.out = k_out;
  vs.out = v_out;
  const int sides = v_cache ? 2 : 1;
  const KvShape sh = kv_shape(num_rows, sides * Hkv, std::max(d, v_cache ? dv : 0), kReadBlocks);
  decltype(&kv_dequantize_kernel<true, 1>) const kerns[2][4] = {
      {kv_dequantize_kernel<false, 1>, kv_dequantize_kernel<false, 2>, kv_dequantize_kernel<false, 3>,
       kv_dequantize_kernel<false, 4>},
      {kv_dequantize_kernel<true, 1>, kv_dequantize_kernel<true, 2>, kv_dequantize_kernel<true, 3>,
       kv_dequantize_kernel<true, 4>}};
  auto kern = kerns[out_is_fp32 ? 1 : 0][sh.chunks - 1];
  kern<<<sh.grid, kKvThreads, 0, stream>>>(ks, vs, sides, num_rows, Hkv, sh.log_l, idx, cache_rows,
                                           status_dev);
  return cudaGetLastError() == cudaSuccess ? CPATTN_OK : CPATTN_ERR_CUDA;
}
