// Attention for a batch that shares keys (cp_attn_shared).
//
// A unit is up to CPATTN_SHARED_ROWS packed rows (query row i, head j of the KV
// head's group, at i*g + j) against one run of keys; the plan cuts the units
// into pieces and gives each thread block a list of them.  A piece's partial
// result per row is (O, L) over its keys,
//     L = ln sum_k exp(S_k),  O = sum_k exp(S_k - L) V_k,
// in fp32; the merge combines a row's partials by the log-sum-exp rule
//     m = max L_j, w_j = exp(L_j - m), O = sum w_j O_j / sum w_j, L = m + ln sum w_j.
#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>

#include "attn_common.cuh"
#include "shared_plan.h"
#include "trace.h"

namespace cpattn {
namespace {

constexpr int kRows = CPATTN_SHARED_ROWS;

struct SharedParams {
  const int32_t* table;
  long long unit_first, row_first, entries, pieces;  // word offsets
  int num_ctas, num_units, num_pieces, num_entries, num_q_rows, Hq, Hkv, g;
  long long ws_rows;
  const __nv_bfloat16* q;
  long long q_row, q_head;
  const void* k;
  const void* v;
  long long k_row, k_head, v_row, v_head;
  const float* ks;
  const float* vs;
  long long s_head;
  int num_kv_rows;
  float scale;
  void* o;
  int o_f32;
  float* lse;
  float* ws_o;
  float* ws_l;
  int32_t* status;
};

// A piece of the table, checked against the buffers; false (and
// CPATTN_ERR_RANGE) when it does not fit them.
__device__ __forceinline__ bool load_piece(const SharedParams& p, int i, SharedPiece& pc) {
  pc = reinterpret_cast<const SharedPiece*>(p.table + p.pieces)[i];
  const bool ok = pc.rows >= 1 && pc.rows <= kRows && pc.r0 >= 0 && pc.q_row0 >= 0 &&
                  (long long)pc.q_row0 + ((long long)pc.r0 + pc.rows - 1) / p.g < p.num_q_rows &&
                  pc.kv_head >= 0 && pc.kv_head < p.Hkv && pc.keys >= 1 && pc.key0 >= 0 &&
                  pc.kv_row >= 0 && (long long)pc.kv_row + pc.keys <= p.num_kv_rows &&
                  pc.ws_row >= 0 && (long long)pc.ws_row + pc.rows <= p.ws_rows;
  if (!ok) set_status(p.status, CPATTN_ERR_RANGE);
  return ok;
}

// One warp per packed row, one key at a time.
template <int D, bool QUANT>
__global__ void __launch_bounds__(512) attn_shared_kernel(const SharedParams p) {
  constexpr int E = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = p.table[blockIdx.x], last = p.table[blockIdx.x + 1];
  if (first < 0 || last > p.num_pieces) {
    set_status(p.status, CPATTN_ERR_RANGE);
    return;
  }
  for (int i = first; i < last; ++i) {
    SharedPiece pc;
    if (!load_piece(p, i, pc)) continue;
    for (int r = warp; r < pc.rows; r += 16) {
      const int packed = pc.r0 + r, qi = packed / p.g, h = pc.kv_head * p.g + packed % p.g;
      const long long pos = (long long)pc.q_pos0 + (long long)qi * pc.q_pos_step;
      const int seen = (int)max(0LL, min((long long)pc.keys, pos + 1 - pc.key0));
      float q[E], acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
      for (int c = 0; c < E; ++c) {
        q[c] = __bfloat162float(p.q[(long long)(pc.q_row0 + qi) * p.q_row + h * p.q_head + lane * E + c]);
        acc[c] = 0.f;
      }
      for (int key = 0; key < seen; ++key) {
        const long long row = pc.kv_row + key;
        const long long ka = row * p.k_row + pc.kv_head * p.k_head + lane * E;
        const long long va = row * p.v_row + pc.kv_head * p.v_head + lane * E;
        float kk[E], vv[E];
#pragma unroll
        for (int c = 0; c < E; ++c) {
          if (QUANT) {
            uint32_t a, b;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"((uint16_t)static_cast<const uint8_t*>(p.k)[ka + c]));
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"((uint16_t)static_cast<const uint8_t*>(p.v)[va + c]));
            const float s1 = p.ks[pc.kv_head * p.s_head + row], s2 = p.vs[pc.kv_head * p.s_head + row];
            float fa, fb;
            asm("cvt.f32.f16 %0, %1;" : "=f"(fa) : "h"((uint16_t)a));
            asm("cvt.f32.f16 %0, %1;" : "=f"(fb) : "h"((uint16_t)b));
            kk[c] = fa * s1;
            vv[c] = fb * s2;
          } else {
            kk[c] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.k)[ka + c]);
            vv[c] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.v)[va + c]);
          }
        }
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < E; ++c) s = fmaf(q[c], kk[c], s);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        s *= p.scale;
        const float mn = fmaxf(m, s);
        const float use = mn == -INFINITY ? 0.f : mn;  // a NaN score stays one
        const float a = expf(m - use), w = expf(s - use);
        l = l * a + w;
#pragma unroll
        for (int c = 0; c < E; ++c) acc[c] = fmaf(acc[c], a, w * vv[c]);
        m = mn;
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int c = 0; c < E; ++c)
        p.ws_o[((long long)pc.ws_row + r) * D + lane * E + c] = acc[c] * inv;
      if (lane == 0) p.ws_l[(long long)pc.ws_row + r] = l == 0.f ? -INFINITY : m + logf(l);
    }
  }
}

// One warp per (query row, head): its partials, in the order of its segments.
template <int D>
__global__ void __launch_bounds__(256) shared_merge_kernel(const SharedParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
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
      const long long row =
          reinterpret_cast<const SharedPiece*>(p.table + p.pieces)[i].ws_row + packed % kRows;
      if (row < 0 || row >= p.ws_rows) {
        if (lane == 0) set_status(p.status, CPATTN_ERR_RANGE);
        return;
      }
      const float lj = p.ws_l[row];
      const float mn = fmaxf(m, lj);
      const float use = mn == -INFINITY ? 0.f : mn;  // a NaN partial stays one
      const float a = expf(m - use), w = expf(lj - use);
      sw = sw * a + w;
#pragma unroll
      for (int c = 0; c < E; ++c) acc[c] = fmaf(acc[c], a, w * p.ws_o[row * D + lane * E + c]);
      m = mn;
    }
  }
  const float inv = sw == 0.f ? 0.f : 1.f / sw;
  const long long out = ((long long)n * p.Hq + h) * D + lane * E;
#pragma unroll
  for (int c = 0; c < E; ++c) {
    if (p.o_f32) static_cast<float*>(p.o)[out + c] = acc[c] * inv;
    else static_cast<__nv_bfloat16*>(p.o)[out + c] = __float2bfloat16_rn(acc[c] * inv);
  }
  if (lane == 0) p.lse[(long long)n * p.Hq + h] = sw == 0.f ? -INFINITY : m + logf(sw);
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
  p.num_ctas = plan->num_ctas;
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
  p.k = k;
  p.v = v;
  p.k_row = k_row_stride;
  p.k_head = k_head_stride;
  p.v_row = v_row_stride;
  p.v_head = v_head_stride;
  p.ks = k_scales;
  p.vs = v_scales;
  p.s_head = scale_stride;
  p.num_kv_rows = num_kv_rows;
  p.scale = scale;
  p.o = o;
  p.o_f32 = o_is_fp32 ? 1 : 0;
  p.lse = lse;
  p.ws_o = static_cast<float*>(workspace);
  p.ws_l = p.ws_o + plan->ws_rows * dv;
  p.status = status_dev;
  if (plan->num_pieces > 0) {
    auto kern = d == 128 ? (quant ? attn_shared_kernel<128, true> : attn_shared_kernel<128, false>)
                         : (quant ? attn_shared_kernel<64, true> : attn_shared_kernel<64, false>);
    kern<<<plan->num_ctas, 512, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return CPATTN_ERR_CUDA;
  }
  const long long blocks = ((long long)plan->num_q_rows * plan->Hq + 7) / 8;
  if (blocks > 0x7fffffffLL) return CPATTN_ERR_TOO_LARGE;
  if (d == 128) shared_merge_kernel<128><<<(unsigned)blocks, 256, 0, stream>>>(p);
  else shared_merge_kernel<64><<<(unsigned)blocks, 256, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? CPATTN_OK : CPATTN_ERR_CUDA;
}
