// Quantised KV cache: write (bf16 / fp32 rows to e4m3 codes with a power-of-two
// scale per row and head) and read back.
//
// For one vector x: a = max finite |x_c|, e = clamp(ceil(log2(a/448)), -117,
// 119), scale = 2^e, code_c = e4m3(x_c 2^-e), value = code_c 2^e.  Both kernels
// are HBM streams: a vector is read once, kept in registers between the maximum
// and the rounding, and its codes are written once.
#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>

#include "../../include/cpattn.h"
#include "ptx.cuh"
#include "trace.h"

namespace cpattn {
namespace {

constexpr int kKvThreads = 256;
constexpr int kMaxDim = 1024;
constexpr int kMinExp = -117, kMaxExp = 119;

// ceil(log2(a / 448)) from the bits of a >= 0: a = m 2^E with m in [1, 2), 448 =
// 1.75 2^8, so it is E - 8, plus one when m > 1.75 (the carry out of the added
// 2^23 - 1 - 0.75 2^23).  A subnormal a comes out below kMinExp.
__device__ __forceinline__ int scale_exponent(float a) {
  const int e = (int)((__float_as_uint(a) + 0x1FFFFFu) >> 23) - 127 - 8;
  return min(max(e, kMinExp), kMaxExp);
}
__device__ __forceinline__ float exp2_int(int e) {  // e in [-126, 127]
  return __uint_as_float((uint32_t)(e + 127) << 23);
}
__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two codes to fp32 (exact: every e4m3 value is an f16).
__device__ __forceinline__ void e4m3x2_to_f32(uint16_t c, float& lo, float& hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}

struct KvSide {  // one of K and V
  const void* x;
  long long x_row, x_head;  // elements
  uint8_t* codes;
  float* scales;
  long long c_row, c_head, s_head;
  void* out;
  int dim;
};

// 8 consecutive elements as fp32.
template <bool F32>
__device__ __forceinline__ void load8(const void* x, long long at, float (&v)[8]) {
  if (F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

// A warp per (row, K or V, head) vector; lane l holds elements 8l.. of each 256.
template <bool F32>
__global__ void __launch_bounds__(kKvThreads)
kv_quantize_kernel(const KvSide k, const KvSide v, int sides, int num_rows, int Hkv,
                   const int32_t* __restrict__ slots, int cache_rows, int32_t* status) {
  const int lane = threadIdx.x & 31;
  const long long vectors = (long long)num_rows * sides * Hkv;
  const long long nwarps = ((long long)gridDim.x * blockDim.x) >> 5;
  for (long long u = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5; u < vectors;
       u += nwarps) {
    const int h = (int)(u % Hkv);
    const long long rs = u / Hkv;
    const KvSide& s = (rs % sides) ? v : k;
    const long long row = rs / sides;
    const int slot = slots ? __ldg(slots + row) : (int)row;
    if (slot < 0 || slot >= cache_rows) {
      if (slot >= 0 && lane == 0) set_status(status, CPATTN_ERR_RANGE);
      continue;
    }
    const long long at = row * s.x_row + (long long)h * s.x_head;
    float x[kMaxDim / 256][8];
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxDim / 256; ++i) {
      const int c = i * 256 + lane * 8;
      if (c < s.dim) {
        load8<F32>(s.x, at + c, x[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float m = fabsf(x[i][j]);
          a = fmaxf(a, m < INFINITY ? m : 0.f);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    const int e = scale_exponent(a);
    const float inv = exp2_int(-e);
    uint8_t* dst = s.codes + (long long)slot * s.c_row + (long long)h * s.c_head;
#pragma unroll
    for (int i = 0; i < kMaxDim / 256; ++i) {
      const int c = i * 256 + lane * 8;
      if (c < s.dim) {
        uint32_t w[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          w[j] = (uint32_t)e4m3x2(x[i][4 * j] * inv, x[i][4 * j + 1] * inv) |
                 (uint32_t)e4m3x2(x[i][4 * j + 2] * inv, x[i][4 * j + 3] * inv) << 16;
        *reinterpret_cast<uint2*>(dst + c) = make_uint2(w[0], w[1]);
      }
    }
    if (lane == 0) s.scales[(long long)h * s.s_head + slot] = exp2_int(e);
  }
}

// A warp per (row, K or V, head) vector.
template <bool F32>
__global__ void __launch_bounds__(kKvThreads)
kv_dequantize_kernel(const KvSide k, const KvSide v, int sides, int num_rows, int Hkv,
                     const int32_t* __restrict__ idx, int cache_rows, int32_t* status) {
  const int lane = threadIdx.x & 31;
  const long long vectors = (long long)num_rows * sides * Hkv;
  const long long nwarps = ((long long)gridDim.x * blockDim.x) >> 5;
  for (long long u = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5; u < vectors;
       u += nwarps) {
    const int h = (int)(u % Hkv);
    const long long rs = u / Hkv;
    const KvSide& s = (rs % sides) ? v : k;
    const long long row = rs / sides;
    const int src = idx ? __ldg(idx + row) : (int)row;
    if (src < 0 || src >= cache_rows) {
      if (src >= 0 && lane == 0) set_status(status, CPATTN_ERR_RANGE);
      continue;
    }
    const float scale = __ldg(s.scales + (long long)h * s.s_head + src);
    const uint8_t* p = s.codes + (long long)src * s.c_row + (long long)h * s.c_head;
    const long long at = (row * Hkv + h) * s.dim;
    for (int c = lane * 8; c < s.dim; c += 256) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(p + c));
      float x[8];
      e4m3x2_to_f32((uint16_t)w.x, x[0], x[1]);
      e4m3x2_to_f32((uint16_t)(w.x >> 16), x[2], x[3]);
      e4m3x2_to_f32((uint16_t)w.y, x[4], x[5]);
      e4m3x2_to_f32((uint16_t)(w.y >> 16), x[6], x[7]);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= scale;
      if (F32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(s.out) + at + c);
        o[0] = make_float4(x[0], x[1], x[2], x[3]);
        o[1] = make_float4(x[4], x[5], x[6], x[7]);
      } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(s.out) + at + c) =
            make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                       pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
      }
    }
  }
}

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Checks one side's cache and moves it into the kernels' form.
int cache_side(const cp_kv_codes_t* c, int dim, int Hkv, int cache_rows, KvSide* s) {
  if (dim < 16 || dim > kMaxDim || dim % 16) return CPATTN_ERR_UNSUPPORTED;
  if (!c->codes || !c->scales) return CPATTN_ERR_INVALID_ARG;
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

unsigned kv_grid(long long vectors) {
  const long long blocks = (vectors * 32 + kKvThreads - 1) / kKvThreads;
  return (unsigned)std::min<long long>(blocks, 1 << 20);
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
  const unsigned grid = kv_grid((long long)num_rows * sides * Hkv);
  auto kern = x_is_fp32 ? kv_quantize_kernel<true> : kv_quantize_kernel<false>;
  kern<<<grid, kKvThreads, 0, stream>>>(ks, vs, sides, num_rows, Hkv, slots, cache_rows,
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
  const unsigned grid = kv_grid((long long)num_rows * sides * Hkv);
  auto kern = out_is_fp32 ? kv_dequantize_kernel<true> : kv_dequantize_kernel<false>;
  kern<<<grid, kKvThreads, 0, stream>>>(ks, vs, sides, num_rows, Hkv, idx, cache_rows, status_dev);
  return cudaGetLastError() == cudaSuccess ? CPATTN_OK : CPATTN_ERR_CUDA;
}
