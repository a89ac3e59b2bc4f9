// Rotary positions, alone (cp_rope) and on the way into a KV cache (cp_kv_append).
//
// Pair c of a vector, (a, b), becomes (a cos t - b sin t, b cos t + a sin t) with the angle
// t = p f_c, p the row's position on the pair's axis; the inverse takes -t.  A position
// times a frequency is up to 2^31 turns, of which fp32 would keep none of the fraction.
// So a frequency is held in turns as a 64-bit fraction F (f / 2 pi mod 1, times 2^64), and
// p F mod 2^64 is the phase, exact but for F's rounding: off by |p| 2^-64 turns at most.  The quarter
// turn next to it is split off before the rest goes to fp32, with all 64 bits, so that cos and sin keep
// fp32's relative bits at any position, those of small angles (slow pairs, first positions) among them.
//
// One kernel for both calls, an HBM stream.  L = 2^k lanes share a vector; a lane's item is
// two 16-byte chunks (of bf16) that hold 8 pairs, or 16 columns that are not rotated.  A
// group of lanes takes vectors of one row, some at a time: it starts their loads, computes
// its part of the block's cos and sin (into shared memory: they serve all heads) while these
// are on their way, and then rotates, rounds or quantises.  Q, K and V have code of their own (one
// code for all, with the side looked up for each vector: 32.1 against 30.3 us).  Measured: 8192
// rows of 40 heads of 128 (bf16) 30.2 us, 5.6 TB/s; fp32 54.8 us, 6.1 TB/s; 4096 rows into an e4m3
// cache 22.7 us; 16384 rows of 576 columns 12.6 us, 3.0 TB/s (a vector is three items of 16 lanes,
// one row a group: what is in flight; with the rows' cos and sin computed by 32 of the threads
// 35.8 us); 64 rows 2.9 us, the launch.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdlib>

#include <cuda_bf16.h>

#include "../../include/cpattn.h"
#include "attn_common.cuh"
#include "kv_codes.cuh"
#include "ptx.cuh"
#include "trace.h"

namespace cpattn {
namespace {

constexpr int kThreads = 256;  // of a block, at most
constexpr int kMaxDim = 1024;
constexpr int kMaxCs = 2048;  // cos and sin values of a block's rows
constexpr int kItem = 16;     // columns of an item

// Vectors that a group of lanes has at a time, as many as 32 to 48 registers hold.
constexpr int units_at_once(bool f32, int items) { return f32 ? (items == 1 ? 2 : 1) : items == 3 ? 1 : 2; }

struct RopeSide {  // Q, K or V; strides in 16 bytes
  const uint8_t* x;
  uint32_t x_row, x_head;
  uint8_t* y;  // codes, or values
  uint32_t y_row, y_head;
  float* scales;  // codes' scales, or null
  long long s_head;
  int heads, dim;
  int cached;   // rows go to their slots, as bf16 or codes; else to their own place, in x's type
};

struct RopeParams {
  RopeSide side[3];
  const int4* table;  // (F low, F high, axis, 0) of each pair
  const int32_t* positions;
  long long axis_stride;
  int pairs, first, axes, inverse;
  const int32_t* slots;
  // vectors of a row; rows of a block; 2^log_l lanes have a vector, 2^log_split groups a row
  int num_rows, cache_rows, vectors, rows, log_l, log_split;
  int32_t* status;
};

// cos and sin of position p times frequency F.
__device__ __forceinline__ float2 cos_sin(int p, uint32_t f_lo, uint32_t f_hi) {
  // in 2^-32 turns, and its low word in 2^-64
  const uint32_t u = (uint32_t)p, phase_lo = u * f_lo, phase = __umulhi(u, f_lo) + u * f_hi - (p < 0 ? f_lo : 0u);
  const uint32_t quarter = (phase + 0x20000000u) >> 30;  // nearest, mod 4
  // The rest, at most half a quarter turn, by its magnitude in two words, of which none cancels: two
  // roundings to fp32, 2^-23 of it (a conversion of all 64 bits costs 0.8 us of 8192 rows' 30).
  const uint32_t up = phase - (quarter << 30), minus = (uint32_t)((int)up >> 31);
  const uint64_t flip = (uint64_t)minus << 32 | minus;
  const uint64_t size = (((uint64_t)up << 32 | phase_lo) ^ flip) - flip;
  const float turns = fmaf((float)(uint32_t)size, 0x1p-63f, (float)(uint32_t)(size >> 32) * 0x1p-31f);
  const float rest = __uint_as_float(__float_as_uint(turns) | (minus & 0x80000000u));  // half turns
  float s, c;
  sincospif(rest, &s, &c);
  const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
  // quarters 0..3: (c, s), (-s, c), (-c, -s), (s, -c)
  return make_float2(quarter == 1 || quarter == 2 ? -a : a, quarter >= 2 ? -b : b);
}

// 8 consecutive elements as they lie in memory, and in fp32.
template <bool F32>
struct Raw8 {
  uint4 v[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const uint8_t* x) {
    const uint4* p = reinterpret_cast<const uint4*>(x);
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) v[i] = __ldcs(p + i);
  }
  __device__ __forceinline__ void values(float* f) const {
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (F32) {
          f[4 * i + j] = __uint_as_float(w[j]);
        } else {
          f[2 * j] = __uint_as_float(w[j] << 16);
          f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
      }
    }
  }
};
__device__ __forceinline__ void store8_bf16(uint8_t* at, const float* f) {
  *reinterpret_cast<uint4*>(at) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                             pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void store8_f32(uint8_t* at, const float* f) {
  reinterpret_cast<float4*>(at)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(at)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void fmul2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void store8_codes(uint8_t* at, const float* f, float inv) {
  uint32_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float x[4];
    fmul2(x[0], x[1], f[4 * j], f[4 * j + 1], inv, inv);
    fmul2(x[2], x[3], f[4 * j + 2], f[4 * j + 3], inv, inv);
    w[j] = (uint32_t)e4m3x2(x[0], x[1]) | (uint32_t)e4m3x2(x[2], x[3]) << 16;
  }
  *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
}

// A group's way through the heads of a side: head h of its row, h + 2^log_split, ...  What a side
// is not (Q and not cached, V and not rotated) falls away in its copy of the code.
template <bool F32, bool INTER, int NI, int SIDE>
struct RopeWalk {
  static constexpr int U = units_at_once(F32, NI), kSize = F32 ? 4 : 2;
  const RopeParams& p;
  const uint8_t* x;
  uint8_t* y;
  float* scale;
  long long x_step, y_step, s_step;
  int h, lane;
  bool live;  // the row is one, and has a place here

  __device__ __forceinline__ const RopeSide& side() const { return p.side[SIDE]; }
  __device__ __forceinline__ bool cached() const { return SIDE == 2 || (SIDE == 1 && side().cached); }
  __device__ __forceinline__ bool rotated() const { return SIDE < 2 && p.pairs > 0; }
  __device__ __forceinline__ bool more() const { return live && h < side().heads; }

  // first: heads of the sides before this one (the vectors of a row are dealt in order).
  __device__ __forceinline__ RopeWalk(const RopeParams& params, int first, int sub, int lane_, uint32_t row, bool live_)
      : p(params), lane(lane_), live(live_) {
    const RopeSide& s = side();
    h = (sub - first) & ((1 << p.log_split) - 1);
    x = s.x + (((unsigned long long)row * s.x_row + (unsigned long long)h * s.x_head) << 4);
    x_step = (long long)s.x_head << (4 + p.log_split);
  }
  // The outputs; slot: the row's place in the caches (looked at here, when loads are on their way).
  __device__ __forceinline__ void place(uint32_t row, int slot) {
    const RopeSide& s = side();
    const int to = cached() ? slot : (int)row;
    if (cached() && (uint32_t)to >= (uint32_t)p.cache_rows) {
      if (live && to >= 0 && lane == 0 && h < s.heads) set_status(p.status, CPATTN_ERR_RANGE);
      live = false;
    }
    y = s.y + (((unsigned long long)(uint32_t)to * s.y_row + (unsigned long long)h * s.y_head) << 4);
    y_step = (long long)s.y_head << (4 + p.log_split);
    if (SIDE > 0) {
      scale = s.scales + (h * s.s_head + to);
      s_step = s.s_head << p.log_split;
    }
  }
  // Columns of item j's chunks.
  __device__ __forceinline__ int2 columns(int j) const {
    if (!rotated()) return make_int2(j * kItem, j * kItem + 8);
    const int eighths = p.pairs / 8;
    if (j < eighths) {
      const int c = p.first + j * (INTER ? 16 : 8);
      return make_int2(c, c + (INTER ? 8 : p.pairs));
    }
    const int n = 2 * (j - eighths), head = p.first / 8;  // chunks before the rotated ones
    return make_int2(8 * (n < head ? n : n + 2 * eighths), 8 * (n + 1 < head ? n + 1 : n + 1 + 2 * eighths));
  }
  __device__ __forceinline__ void load(Raw8<F32> (&raw)[U][NI][2]) const {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int j = lane + (i << p.log_l);
        if (!live || h + (u << p.log_split) >= side().heads || j * kItem >= side().dim) continue;
        const int2 c = columns(j);
        raw[u][i][0].load(x + u * x_step + c.x * kSize);
        raw[u][i][1].load(x + u * x_step + c.y * kSize);
      }
  }
  // cs: cos and sin of the row (see the kernel); keep: those of a lane's one item.
  __device__ __forceinline__ void store(const Raw8<F32> (&raw)[U][NI][2], const float4* cs, const float4 (&keep)[4],
                                        uint32_t mask) {
    const RopeSide& s = side();
    const int eighths = p.pairs / 8;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!live || h + (u << p.log_split) >= s.heads) continue;  // (the same in the vector's lanes)
      float f[NI][kItem];
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        raw[u][i][0].values(f[i]);
        raw[u][i][1].values(f[i] + 8);
        const int j = lane + (i << p.log_l);
        if (!rotated() || j >= eighths) continue;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 v = NI == 1 ? keep[k] : cs[k * eighths + j];
          float& a0 = f[i][INTER ? 4 * k : 2 * k];
          float& a1 = f[i][INTER ? 4 * k + 2 : 2 * k + 1];
          float& b0 = f[i][INTER ? 4 * k + 1 : 2 * k + 8];
          float& b1 = f[i][INTER ? 4 * k + 3 : 2 * k + 9];
          float ac0, ac1, bc0, bc1;
          fmul2(ac0, ac1, a0, a1, v.x, v.y);
          fmul2(bc0, bc1, b0, b1, v.x, v.y);
          ffma2(bc0, bc1, a0, a1, v.z, v.w, bc0, bc1);
          ffma2(a0, a1, b0, b1, -v.z, -v.w, ac0, ac1);
          b0 = bc0;
          b1 = bc1;
        }
      }
      const bool codes = SIDE > 0 && s.scales;
      float inv = 1.f;
      if (codes) {
        // the largest finite element; the rotated value is rounded once, to its code
        auto largest = [&](bool finite) {
          float a = 0.f;
#pragma unroll
          for (int i = 0; i < NI; ++i)
            if ((lane + (i << p.log_l)) * kItem < s.dim)
#pragma unroll
              for (int e = 0; e < kItem; ++e) {
                const float m = fabsf(f[i][e]);
                a = fmaxf(a, !finite || m < INFINITY ? m : 0.f);
              }
          for (int o = 1 << p.log_l >> 1; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(mask, a, o));
          return a;
        };
        float a = largest(false);
        if (a == INFINITY) a = largest(true);  // (fmaxf leaves a NaN out by itself)
        const int e = scale_exponent(a);
        inv = exp2_int(-e);
        if (lane == 0) scale[u * s_step] = exp2_int(e);
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int j = lane + (i << p.log_l);
        if (j * kItem >= s.dim) continue;
        const int2 c = columns(j);
        uint8_t* const at = y + u * y_step;
        if (codes) {
          store8_codes(at + c.x, f[i], inv);
          store8_codes(at + c.y, f[i] + 8, inv);
        } else if (F32 && !cached()) {
          store8_f32(at + 4 * c.x, f[i]);
          store8_f32(at + 4 * c.y, f[i] + 8);
        } else {
          store8_bf16(at + 2 * c.x, f[i]);
          store8_bf16(at + 2 * c.y, f[i] + 8);
        }
      }
    }
    h += U << p.log_split;
    x += U * x_step;
    y += U * y_step;
    if (SIDE > 0) scale += U * s_step;
  }
};

// NI: items of a lane.  INTER: pairs are neighbours (a rotated item's chunks then lie
// side by side); else (c, c + pairs).
template <bool F32, bool INTER, int NI>
__global__ void __launch_bounds__(kThreads, NI != 1 || F32 ? 2 : 3) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int U = units_at_once(F32, NI);
  // (c, c', s, s') of pairs 8 j + 2 k, 8 j + 2 k + 1 of row r at [r][k][j]: lanes j side by side
  __shared__ float4 cs[kMaxCs / 2];
  const int L = 1 << p.log_l, lane = threadIdx.x & (L - 1), group = threadIdx.x >> p.log_l;
  const uint32_t mask = (L == 32 ? 0xffffffffu : (1u << L) - 1u) << (threadIdx.x & 31 & ~(L - 1));
  const int h0 = p.side[0].heads, h1 = h0 + p.side[1].heads, eighths = p.pairs / 8;
  const long long r0 = (long long)blockIdx.x * p.rows;
  const int sub = group & ((1 << p.log_split) - 1), r = group >> p.log_split;
  const int rows = (int)min((long long)p.rows, p.num_rows - r0);
  const bool live = r < rows;
  const uint32_t row = (uint32_t)(r0 + (live ? r : 0));
  // the row's place in the caches
  const int slot = live && p.slots ? __ldg(p.slots + row) : (int)row;
  RopeWalk<F32, INTER, NI, 0> q(p, 0, sub, lane, row, live);
  RopeWalk<F32, INTER, NI, 1> k(p, h0, sub, lane, row, live);
  Raw8<F32> raw[U][NI][2];
  if (h0 > 0) q.load(raw);
  else k.load(raw);
  if (p.pairs > 0) {
    for (int i = threadIdx.x; i < rows * p.pairs; i += blockDim.x) {
      const int at_row = i / p.pairs, c = i - at_row * p.pairs;
      const int4 f = __ldg(p.table + c);
      const bool ok = f.z >= 0 && f.z < p.axes;
      if (!ok) set_status(p.status, CPATTN_ERR_RANGE);
      const int at = ok ? __ldg(p.positions + f.z * p.axis_stride + r0 + at_row) : 0;
      const float2 v = cos_sin(at, (uint32_t)f.x, (uint32_t)f.y);
      float* const dst = reinterpret_cast<float*>(cs + (at_row * 4 + ((c >> 1) & 3)) * eighths + (c >> 3)) + (c & 1);
      dst[0] = v.x;
      dst[2] = p.inverse ? -v.y : v.y;
    }
    __syncthreads();
  }
  const float4* const mine = cs + r * 4 * eighths;
  float4 keep[4];
  if (NI == 1 && live && lane < eighths)
#pragma unroll
    for (int x = 0; x < 4; ++x) keep[x] = mine[x * eighths + lane];
  k.place(row, slot);
  if (h0 > 0) {
    q.place(row, slot);
    while (q.more()) {
      q.store(raw, mine, keep, mask);
      if (q.more()) q.load(raw);
    }
    if (k.more()) k.load(raw);
  }
  while (k.more()) {
    k.store(raw, mine, keep, mask);
    if (k.more()) k.load(raw);
  }
  if (p.side[2].heads > 0) {
    RopeWalk<F32, INTER, NI, 2> v(p, h1, sub, lane, row, live);
    v.place(row, slot);
    while (v.more()) {
      v.load(raw);
      v.store(raw, mine, keep, mask);
    }
  }
}

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Rows [n, heads, dim] with strides in elements of `size` bytes, 16-byte aligned.
int check_rows(const void* x, int64_t row, int64_t head, int size) {
  if (!aligned(x, 16) || row % (16 / size) || head % (16 / size)) return CPATTN_ERR_ALIGNMENT;
  return row < 0 || head < 0 ? CPATTN_ERR_INVALID_ARG : CPATTN_OK;
}
// ... that are written: no element has two places.
int check_out_rows(const void* x, int64_t row, int64_t head, int size, int64_t n, int heads, int dim) {
  const int rc = check_rows(x, row, head, size);
  if (rc != CPATTN_OK) return rc;
  if (n == 0) return CPATTN_OK;
  const bool by_row = (heads == 1 || head >= dim) && (n == 1 || row >= (heads - 1) * head + dim);
  const bool by_head = (n == 1 || row >= dim) && (heads == 1 || head >= (n - 1) * row + dim);
  return by_row || by_head ? CPATTN_OK : CPATTN_ERR_INVALID_ARG;
}
// Whether an output lies apart from its input, or on it with equal strides (each lane
// reads what it writes).  In rows of equal strides the two may lie side by side, with equal strides of
// heads also between each other.
bool apart(const void* x, int64_t xr, int64_t xh, const void* y, int64_t yr, int64_t yh, int size, int64_t n,
           int heads, int dim) {
  if (n == 1) xr = yr = 0;
  if (heads == 1) xh = yh = 0;
  if (x == y && xr == yr && xh == yh) return true;
  const intptr_t a = reinterpret_cast<intptr_t>(x), b = reinterpret_cast<intptr_t>(y);
  const int64_t wx = ((heads - 1) * xh + dim) * size, wy = ((heads - 1) * yh + dim) * size;  // of a row
  if (a + (n - 1) * xr * size + wx <= b || b + (n - 1) * yr * size + wy <= a) return true;
  const int64_t row = xr * size, width = (int64_t)dim * size;
  if (xr != yr) return false;
  if (row > 0) {  // side by side in the rows of one buffer
    const int64_t at = ((b - a) % row + row) % row;
    if (at >= wx && at + wy <= row) return true;
  }
  if (xh != yh) return false;
  // a vector of y, i rows and j heads further on than one of x, that would lie on it
  for (int64_t j = 1 - heads; j < heads; ++j) {
    const int64_t at = b - a + j * xh * size, i0 = row > 0 ? -at / row : 0;
    for (int64_t i = std::max(i0 - 1, 1 - n); i <= std::min(i0 + 1, n - 1); ++i)
      if (std::llabs(at + i * row) < width) return false;
  }
  return true;
}

int check_rope(const cp_rope_t* r, int d, const int32_t* positions, int64_t axis_stride, int num_rows) {
  if (r->pairs < 1 || r->first < 0 || r->axes < 1 || r->axes > CPATTN_MAX_ROPE_AXES) return CPATTN_ERR_INVALID_ARG;
  if (r->pairs % 8 || r->first % 8) return CPATTN_ERR_UNSUPPORTED;
  if ((long long)r->first + 2LL * r->pairs > d) return CPATTN_ERR_INVALID_ARG;
  if (!aligned(r->table, 16) || !aligned(positions, 4)) return CPATTN_ERR_ALIGNMENT;
  if (num_rows > 0 && (!r->table || !positions)) return CPATTN_ERR_INVALID_ARG;
  return r->axes > 1 && axis_stride < 0 ? CPATTN_ERR_INVALID_ARG : CPATTN_OK;
}

int launch_rope(RopeParams& p, const cp_rope_t* rope, bool f32, cudaStream_t stream) {
  const bool inter = rope && rope->interleaved;
  int dim = 0;
  p.vectors = 0;
  for (int i = 0; i < 3; ++i) {
    if (!p.side[i].heads) continue;
    p.vectors += p.side[i].heads;
    dim = std::max(dim, p.side[i].dim);
  }
  if (p.vectors == 0) return CPATTN_OK;
  if (rope) {
    p.table = reinterpret_cast<const int4*>(rope->table);
    p.pairs = rope->pairs;
    p.first = rope->first;
    p.axes = rope->axes;
  }
  // Lanes of a vector: one item each where 32 are enough; 33 to 48 items (576 columns: 36)
  // in three rounds of 16 lanes leave fewer idle than two of 32.
  const int items = dim / kItem;
  int ni = 1;
  if (items > 48) p.log_l = 5, ni = 2;
  else if (items > 32) p.log_l = 4, ni = 3;
  else
    for (p.log_l = 0; (1 << p.log_l) < items; ++p.log_l) {}
  // Blocks of 128 threads, whose share of the last wave is smaller than that of 256 (8192 rows
  // of 40 heads 34.7 -> 33.7 us, 16384 rows of 576 columns 13.5 -> 12.3); of 256 where a
  // block for each row is on the SMs at once: more threads to a row are sooner through (400 rows
  // of 48: 3.6 against 4.0 us; 500 rows, a second wave, 5.1 against 4.1).
  const int log_threads = p.num_rows <= 152 * 3 ? 8 : 7, log_groups = log_threads - p.log_l;
  // Groups of a row: few, since they share its cos and sin, but so many that there are 18
  // blocks for each SM (8192 rows: 33.7 us with half as many, 32.4 with these), and six even if
  // a group then has less than two rounds of vectors (4096 rows of 48: 23.8 us, with twice as
  // many groups 24.6).
  p.log_split = 0;
  while (p.log_split < log_groups && (1 << p.log_split) < p.vectors &&
         ((long long)p.num_rows << p.log_split >> log_groups) <
             (p.vectors >> (p.log_split + 1) >= 4 ? 152 * 18 : 152 * 6))
    ++p.log_split;
  while (p.pairs << (log_groups - p.log_split) > kMaxCs) ++p.log_split;  // (its cos and sin fit: a row has at most 512)
  p.rows = 1 << (log_groups - p.log_split);
  const unsigned grid = (unsigned)(((long long)p.num_rows + p.rows - 1) / p.rows);
  decltype(&rope_kernel<true, true, 1>) const kerns[2][2][3] = {
      {{rope_kernel<false, false, 1>, rope_kernel<false, false, 2>, rope_kernel<false, false, 3>},
       {rope_kernel<false, true, 1>, rope_kernel<false, true, 2>, rope_kernel<false, true, 3>}},
      {{rope_kernel<true, false, 1>, rope_kernel<true, false, 2>, rope_kernel<true, false, 3>},
       {rope_kernel<true, true, 1>, rope_kernel<true, true, 2>, rope_kernel<true, true, 3>}}};
  kerns[f32 ? 1 : 0][inter ? 1 : 0][ni - 1]<<<grid, 1 << log_threads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? CPATTN_OK : CPATTN_ERR_CUDA;
}

// Strides in bytes to those in 16 bytes, of 32 bits (the one row's or head's is not used).
int strides16(RopeSide* s, int64_t xr, int64_t xh, int64_t yr, int64_t yh, int rows, int heads) {
  if (rows <= 1) xr = yr = 0;
  if (heads == 1) xh = yh = 0;
  if (std::max(std::max(xr, xh), std::max(yr, yh)) / 16 > 0xffffffffLL) return CPATTN_ERR_TOO_LARGE;
  s->x_row = (uint32_t)(xr / 16);
  s->x_head = (uint32_t)(xh / 16);
  s->y_row = (uint32_t)(yr / 16);
  s->y_head = (uint32_t)(yh / 16);
  return CPATTN_OK;
}

// One rotated tensor of cp_rope, or Q of cp_kv_append.
int rotated_side(RopeSide* s, const void* x, int64_t xr, int64_t xh, int heads, void* y, int64_t yr, int64_t yh,
                 bool f32, int num_rows, int d) {
  const int size = f32 ? 4 : 2;
  int rc = check_rows(x, xr, xh, size);
  if (rc == CPATTN_OK) rc = check_out_rows(y, yr, yh, size, num_rows, heads, d);
  if (rc != CPATTN_OK) return rc;
  if (num_rows > 0 && (!x || !y)) return CPATTN_ERR_INVALID_ARG;
  if (num_rows > 0 && !apart(x, xr, xh, y, yr, yh, size, num_rows, heads, d)) return CPATTN_ERR_INVALID_ARG;
  s->x = static_cast<const uint8_t*>(x);
  s->y = static_cast<uint8_t*>(y);
  s->heads = heads;
  s->dim = d;
  return strides16(s, xr * size, xh * size, yr * size, yh * size, num_rows, heads);
}

// K or V of cp_kv_append.
int cached_side(RopeSide* s, const void* x, int64_t xr, int64_t xh, bool f32, int heads, int dim,
                const cp_kv_codes_t* c, int num_rows, int cache_rows) {
  const int rc = check_rows(x, xr, xh, f32 ? 4 : 2);
  if (rc != CPATTN_OK) return rc;
  if (dim < 16 || dim > kMaxDim || dim % 16) return CPATTN_ERR_UNSUPPORTED;
  const int size = c->scales ? 1 : 2;
  if ((num_rows > 0 && !x) || (cache_rows > 0 && !c->codes)) return CPATTN_ERR_INVALID_ARG;
  if (!aligned(c->codes, 16) || !aligned(c->scales, 4) || c->row_stride % 16 || c->head_stride % 16)
    return CPATTN_ERR_ALIGNMENT;
  if (c->head_stride < (int64_t)dim * size || c->row_stride < (int64_t)(heads - 1) * c->head_stride + dim * size ||
      (c->scales && c->scale_stride < cache_rows))
    return CPATTN_ERR_INVALID_ARG;
  s->x = static_cast<const uint8_t*>(x);
  s->y = static_cast<uint8_t*>(c->codes);
  s->scales = c->scales;
  s->s_head = c->scale_stride;
  s->heads = heads;
  s->dim = dim;
  s->cached = 1;
  const int in = f32 ? 4 : 2;
  return strides16(s, xr * in, xh * in, c->row_stride, c->head_stride, std::max(num_rows, cache_rows), heads);
}

}  // namespace
}  // namespace cpattn

using namespace cpattn;

extern "C" int cp_rope_table(const double* inv_freq, const int32_t* axis, int pairs, int32_t* table) {
  if (!inv_freq || !table || pairs < 1 || pairs > kMaxDim / 2) return CPATTN_ERR_INVALID_ARG;
  // 1 / (2 pi) in two parts, so that the product keeps 2^-64 of a turn
  const double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
  for (int c = 0; c < pairs; ++c) {
    const double f = inv_freq[c];
    const int a = axis ? axis[c] : 0;
    if (!(std::fabs(f) <= 0x1p20) || a < 0 || a >= CPATTN_MAX_ROPE_AXES) return CPATTN_ERR_INVALID_ARG;
    const double turns = f * hi, rest = std::fma(f, hi, -turns) + f * lo;
    // in 2^-64 turns, of a turn's fraction: that part is exact for either sign (turns - floor(turns) is
    // not below zero), and so is its split at the binary point, so that one rounding is left
    const double part = std::ldexp(turns - std::trunc(turns), 64), whole = std::trunc(part);
    const uint64_t up = (uint64_t)std::fabs(whole);
    const uint64_t F = (whole < 0 ? 0 - up : up) + (uint64_t)std::llrint(std::ldexp(rest, 64) + (part - whole));
    table[4 * c] = (int32_t)(uint32_t)F;
    table[4 * c + 1] = (int32_t)(uint32_t)(F >> 32);
    table[4 * c + 2] = a;
    table[4 * c + 3] = 0;
  }
  return CPATTN_OK;
}

extern "C" int cp_rope(const cp_rope_t* rope, const cp_rope_args_t* a, cudaStream_t stream) {
  CPATTN_TRACE("cp_rope");
  if (!rope || !a || a->num_rows < 0 || a->Hq < 1 || a->Hk < 0 || a->Hq > 1 << 20 || a->Hk > 1 << 20)
    return CPATTN_ERR_INVALID_ARG;
  if (a->d < 16 || a->d > kMaxDim || a->d % 16) return CPATTN_ERR_UNSUPPORTED;
  if (!aligned(a->status_dev, 4)) return CPATTN_ERR_ALIGNMENT;
  int rc = check_rope(rope, a->d, a->positions, a->axis_stride, a->num_rows);
  if (rc != CPATTN_OK) return rc;
  RopeParams p{};
  const bool f32 = a->x_is_fp32 != 0;
  rc = rotated_side(&p.side[0], a->q, a->q_row_stride, a->q_head_stride, a->Hq, a->q_out, a->qo_row_stride,
                    a->qo_head_stride, f32, a->num_rows, a->d);
  if (rc == CPATTN_OK && a->Hk > 0)
    rc = rotated_side(&p.side[1], a->k, a->k_row_stride, a->k_head_stride, a->Hk, a->k_out, a->ko_row_stride,
                      a->ko_head_stride, f32, a->num_rows, a->d);
  if (rc != CPATTN_OK || a->num_rows == 0) return rc;
  p.positions = a->positions;
  p.axis_stride = a->axis_stride;
  p.inverse = a->inverse ? 1 : 0;
  p.num_rows = a->num_rows;
  p.status = a->status_dev;
  return launch_rope(p, rope, f32, stream);
}

extern "C" int cp_kv_append(const cp_rope_t* rope, const cp_kv_codes_t* k_cache, const cp_kv_codes_t* v_cache,
                            const cp_kv_append_args_t* a, cudaStream_t stream) {
  CPATTN_TRACE("cp_kv_append");
  if (!a || a->num_rows < 0 || a->cache_rows < 0 || a->Hkv < 1 || a->Hkv > 1 << 20 || a->Hq < 0 || a->Hq > 1 << 20 ||
      !k_cache || (a->v && !v_cache) || (a->num_rows > 0 && !a->v && v_cache) ||
      (v_cache && !v_cache->scales != !k_cache->scales))
    return CPATTN_ERR_INVALID_ARG;
  if (!aligned(a->slots, 4) || !aligned(a->status_dev, 4)) return CPATTN_ERR_ALIGNMENT;
  int rc = rope ? check_rope(rope, a->d, a->positions, a->axis_stride, a->num_rows) : CPATTN_OK;
  if (rc != CPATTN_OK) return rc;
  RopeParams p{};
  const bool f32 = a->x_is_fp32 != 0;
  rc = cached_side(&p.side[1], a->k, a->k_row_stride, a->k_head_stride, f32, a->Hkv, a->d, k_cache, a->num_rows,
                   a->cache_rows);
  if (rc == CPATTN_OK && v_cache)
    rc = cached_side(&p.side[2], a->v, a->v_row_stride, a->v_head_stride, f32, a->Hkv, a->dv, v_cache, a->num_rows,
                     a->cache_rows);
  if (rc == CPATTN_OK && a->Hq > 0)
    rc = rotated_side(&p.side[0], a->q, a->q_row_stride, a->q_head_stride, a->Hq, a->q_out, a->qo_row_stride,
                      a->qo_head_stride, f32, a->num_rows, a->d);
  if (rc != CPATTN_OK || a->num_rows == 0) return rc;
  p.positions = a->positions;
  p.axis_stride = a->axis_stride;
  p.slots = a->slots;
  p.num_rows = a->num_rows;
  p.cache_rows = a->cache_rows;
  p.status = a->status_dev;
  return launch_rope(p, rope, f32, stream);
}
