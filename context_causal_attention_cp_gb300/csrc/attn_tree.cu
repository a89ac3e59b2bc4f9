// Attention of new rows (single tokens, chains, trees of drafted tokens) over a paged cache
// (cp_attn_tree): the merge of cut units, and the host's part.
#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>

#include "attn_tree.cuh"
#include "trace.h"

namespace cpattn {
namespace {

// Merge of the units that the blocks' shares cut: blocks (x, y) take the unit that is cut behind
// attention block x.  A row's partials (O_j, L_j) combine as
//     m = max L_j, w_j = exp(L_j - m), O = sum w_j O_j / sum w_j, L = m + ln sum w_j.
// Bound by latency, two dependent loads: the unit's description, and then L and O of up to
// `LOADS` partials at once.  A thread has 4 columns of a row; where a unit has fewer values
// than the block threads, several share a value's partials and are joined in shared memory.
// Units of 8 and 16 rows: 512 threads, 8 loads; those of 128 and 256, of which most are cut
// once, 256 and 4, for their bytes.
struct MergeValue {  // sum_j 2^(L_j - m) (1, O_j)
  float m, w;
  float4 o;
};
__device__ __forceinline__ void merge_add(MergeValue& a, float m, float w, const float4& o) {
  const float mn = fmaxf(a.m, m), use = mn == -INFINITY ? 0.f : mn;
  const float fa = exp2f(a.m - use), fb = exp2f(m - use);
  a.m = mn;
  a.w = a.w * fa + w * fb;  // (a NaN partial stays one)
  // (nothing of a partial without keys, whose O is zeros)
  a.o = make_float4(a.o.x * fa + o.x * fb, a.o.y * fa + o.y * fb, a.o.z * fa + o.z * fb, a.o.w * fa + o.w * fb);
}
template <int D, int THREADS, int LOADS>
__global__ void __launch_bounds__(THREADS) tree_merge_kernel(const TreeParams p) {
  __shared__ MergeValue part[THREADS];
  grid_dep_wait();
  const int4 a = __ldcg(p.cut + 2 * blockIdx.x);
  const int blocks = __ldcg(p.cut + 2 * blockIdx.x + 1).x;
  if (blocks < 2 || (long long)blockIdx.x + (blocks - 1LL) * p.team >= gridDim.x) return;
  const int R = p.unit_rows, rows = a.z, values = rows * (D / 4);
  int ways = 1;
  while (ways < blocks && 2 * ways * values <= THREADS) ways *= 2;
  const int way = ways == 1 ? 0 : (int)threadIdx.x / values;
  auto slot_of = [&](int j) { return 2 * ((int)blockIdx.x + j * p.team) + (j == 0 ? 1 : 0); };
  for (int i0 = blockIdx.y * THREADS; i0 < values; i0 += gridDim.y * THREADS) {
    // half a chunk of 8 columns of a row
    const int i = ways == 1 ? i0 + (int)threadIdx.x : (int)threadIdx.x - way * values;
    const bool on = i < values && way < ways;
    const int half = i & 1, c = (i >> 1) / rows, r = (i >> 1) - c * rows;
    MergeValue v{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int j0 = way; on && j0 < blocks; j0 += ways * LOADS) {
      float l[LOADS];
      float4 o[LOADS];
#pragma unroll
      for (int x = 0; x < LOADS; ++x) {
        const int j = j0 + x * ways;
        l[x] = -INFINITY;
        o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j < blocks) {
          const long long slot = (long long)slot_of(j) * R;
          l[x] = __ldcg(p.ws_l + slot + r);
          o[x] = __ldcg(reinterpret_cast<const float4*>(p.ws_o + slot * D + partial_at(c, r, R)) + half);
        }
      }
#pragma unroll
      for (int x = 0; x < LOADS; ++x)
        if (j0 + x * ways < blocks) merge_add(v, l[x], l[x] == -INFINITY ? 0.f : 1.f, o[x]);
    }
    if (ways > 1) {  // (one round)
      part[threadIdx.x] = v;
      __syncthreads();
      if (way > 0 || !on) return;
      for (int y = 1; y < ways; ++y) {
        const MergeValue& other = part[threadIdx.x + y * values];
        merge_add(v, other.m, other.w, other.o);
      }
    }
    if (!on) continue;
    const float inv = v.w == 0.f ? 0.f : 1.f / v.w;
    const float4 out = make_float4(v.o.x * inv, v.o.y * inv, v.o.z * inv, v.o.w * inv);
    const int packed = a.y + r, node = group_div(p, packed);
    const long long at = (long long)(a.x + node) * p.Hq + a.w * p.g + packed - node * p.g;
    const int col = c * 8 + half * 4;
    if (p.o_f32)
      *reinterpret_cast<float4*>(static_cast<float*>(p.o) + at * D + col) = out;
    else
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + at * D + col) =
          make_uint2(pack_bf16x2(out.x, out.y), pack_bf16x2(out.z, out.w));
    if (col == 0) p.lse[at] = v.w == 0.f ? -INFINITY : (v.m + log2f(v.w)) * kLn2;
  }
}

template <int D, int THREADS, int LOADS>
cudaError_t launch_merge(const TreeParams& p, int num_ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_ctas, (p.unit_rows * (D / 4) + THREADS - 1) / THREADS);
  cfg.blockDim = dim3(THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, THREADS, LOADS>, p);
}
template <int D>
cudaError_t launch_merge(const TreeParams& p, int num_ctas, cudaStream_t stream) {
  return p.unit_rows < BM ? launch_merge<D, 512, 8>(p, num_ctas, stream) : launch_merge<D, 256, 4>(p, num_ctas, stream);
}

// 3-D map of a cache (cols, heads, rows) with a box of one head and 64 columns (codes: all). A
// head's row is all that a block reads of a cache row, so that L2 must not fetch more of it:
// with 256 bytes at a time, the 128 of a head's codes brought another head's along.
bool make_rows_map(CUtensorMap* m, const void* base, int cols, bool codes, int heads, long long rows,
                   int64_t head_stride, int64_t row_stride, int box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const int size = codes ? 1 : 2, bytes = cols * size;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)(head_stride * size), (cuuint64_t)(row_stride * size)};
  cuuint32_t box[3] = {(cuuint32_t)(codes ? cols : 64), 1, (cuuint32_t)box_rows};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             bytes == 64    ? CU_TENSOR_MAP_L2_PROMOTION_L2_64B
             : bytes == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                            : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3-D map of the queries (cols, heads, rows) whose box is 64 columns of the g heads of a KV
// head and of BM / g rows.
bool make_q_map(CUtensorMap* m, const void* q, int cols, int heads, int rows, int64_t head_stride,
                int64_t row_stride, int g) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)(head_stride * 2), (cuuint64_t)(row_stride * 2)};
  cuuint32_t box[3] = {64, (cuuint32_t)g, (cuuint32_t)(BM / g)};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Blocks of a team: a divisor of the KV heads, the largest up to 8 that leaves few blocks (a
// fiftieth) without a team.
int team_of(int Hkv, int num_ctas) {
  int team = 1;
  for (int t = 2; t <= 8; ++t)
    if (Hkv % t == 0 && t <= num_ctas && num_ctas % t <= num_ctas / 50) team = t;
  return team;
}

// Packed rows of a unit, by the rows that a request is expected to have.
int unit_rows_of(int g, int max_nodes) {
  const long long rows = (long long)g * max_nodes;
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= BM ? BM : 2 * BM;
}

// Where the parts of a workspace lie, and its size.
void plan_sizes(int Hq, int Hkv, int dv, int max_nodes, int num_ctas, int* unit_rows, int64_t* o_at, int64_t* l_at,
                int64_t* bytes) {
  *unit_rows = unit_rows_of(Hq / Hkv, max_nodes);
  const int64_t rows = 2LL * num_ctas * *unit_rows;
  *o_at = 32LL * num_ctas;  // behind the cut units
  *l_at = *o_at + rows * dv * 4;
  *bytes = (*l_at + rows * 4 + 31) & ~31LL;
}

}  // namespace
}  // namespace cpattn

using namespace cpattn;

extern "C" int cp_tree_workspace_size(int Hq, int Hkv, int dv, int max_nodes, int num_ctas, int64_t* bytes) {
  if (!bytes || Hkv < 1 || Hq < Hkv || Hq % Hkv || Hq > 1 << 20 || max_nodes < 1 || num_ctas < 1 || num_ctas > 4096)
    return CPATTN_ERR_INVALID_ARG;
  if (dv != 64 && dv != 128) return CPATTN_ERR_UNSUPPORTED;
  int rows;
  int64_t o_at, l_at;
  plan_sizes(Hq, Hkv, dv, max_nodes, num_ctas, &rows, &o_at, &l_at, bytes);
  return CPATTN_OK;
}

extern "C" int cp_attn_tree(const cp_attn_tree_args_t* a, cudaStream_t stream) {
  CPATTN_TRACE("cp_attn_tree");
  if (!a) return CPATTN_ERR_INVALID_ARG;
  int64_t need = 0;
  const int rc = cp_tree_workspace_size(a->Hq, a->Hkv, a->dv, a->max_nodes, a->num_ctas, &need);
  if (rc != CPATTN_OK) return rc;
  const int d = a->d, Hkv = a->Hkv, page = a->page_size;
  if (d != a->dv) return CPATTN_ERR_UNSUPPORTED;
  if (page < 16 || page > 65536 || (page & (page - 1))) return CPATTN_ERR_UNSUPPORTED;
  if (!(a->scale > 0.f) || a->num_rows < 0 || a->num_kv_rows < 0 || a->num_reqs < 0 ||
      a->num_reqs > CPATTN_MAX_REQS || a->max_pages < 0 || a->mask_words < 0 ||
      (a->mask != nullptr) != (a->mask_words > 0) || (a->k_scales != nullptr) != (a->v_scales != nullptr) ||
      (a->num_reqs > 1 && a->table_stride < a->max_pages))
    return CPATTN_ERR_INVALID_ARG;
  if ((long long)a->num_rows * (a->Hq / Hkv) > 0x7fffffffLL - CPATTN_SHARED_ROWS) return CPATTN_ERR_TOO_LARGE;
  if (a->num_rows == 0 || a->num_reqs == 0) return CPATTN_OK;  // nothing to write
  if (!a->q || !a->k || !a->v || !a->page_table || !a->q_start || !a->kv_lens || !a->o || !a->lse || !a->workspace ||
      a->workspace_bytes < need || a->num_kv_rows < page || a->max_pages < 1)
    return CPATTN_ERR_INVALID_ARG;
  const bool quant = a->k_scales != nullptr;
  const int64_t per16 = quant ? 16 : 8;  // elements in 16 bytes
  if (!a16(a->q) || !a16(a->k) || !a16(a->v) || !a16(a->o) || (reinterpret_cast<uintptr_t>(a->workspace) & 31u) ||
      a->q_row_stride % 8 || a->q_head_stride % 8 || a->k_row_stride % per16 || a->k_head_stride % per16 ||
      a->v_row_stride % per16 || a->v_head_stride % per16)
    return CPATTN_ERR_ALIGNMENT;
  for (const void* at : {(const void*)a->k_scales, (const void*)a->v_scales, (const void*)a->page_table,
                         (const void*)a->q_start, (const void*)a->kv_lens, (const void*)a->mask, (const void*)a->lse,
                         (const void*)a->status_dev})
    if (reinterpret_cast<uintptr_t>(at) & 3u) return CPATTN_ERR_ALIGNMENT;
  if (a->q_row_stride < 0 || a->q_head_stride < 0 || a->k_head_stride < d || a->v_head_stride < d ||
      a->k_row_stride < (int64_t)(Hkv - 1) * a->k_head_stride + d ||
      a->v_row_stride < (int64_t)(Hkv - 1) * a->v_head_stride + d || (quant && a->scale_stride < a->num_kv_rows))
    return CPATTN_ERR_INVALID_ARG;

  TreeParams p{};
  p.q_start = a->q_start;
  p.kv_lens = a->kv_lens;
  p.page_table = a->page_table;
  p.mask = a->mask;
  p.table_stride = a->table_stride;
  p.num_reqs = a->num_reqs;
  p.num_rows = a->num_rows;
  p.max_pages = a->max_pages;
  for (p.log_page = 4; (1 << p.log_page) < page; ++p.log_page) {}
  p.words = a->mask_words;
  p.Hq = a->Hq;
  p.Hkv = Hkv;
  p.g = a->Hq / Hkv;
  for (p.g_shift = 0; (1LL << (p.g_shift + 1)) < p.g; ++p.g_shift) {}  // see group_div
  p.g_mul = (uint32_t)((1ULL << (32 + p.g_shift)) / p.g + 1);
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  p.q_row = a->q_row_stride;
  p.q_head = a->q_head_stride;
  p.ks = a->k_scales;
  p.vs = a->v_scales;
  p.s_head = a->scale_stride;
  p.scales_16 = a16(a->k_scales) && a16(a->v_scales) && (a->scale_stride % 4 == 0 || Hkv == 1);
  p.num_kv_rows = a->num_kv_rows;
  p.scale_log2 = a->scale * kLog2e;
  p.o = a->o;
  p.o_f32 = a->o_is_fp32 ? 1 : 0;
  p.o_32 = (reinterpret_cast<uintptr_t>(a->o) & 31u) == 0;
  p.lse = a->lse;
  int64_t o_at, l_at, bytes;
  plan_sizes(a->Hq, Hkv, d, a->max_nodes, a->num_ctas, &p.unit_rows, &o_at, &l_at, &bytes);
  while ((1 << p.unit_log) < p.unit_rows) ++p.unit_log;
  p.team = team_of(Hkv, a->num_ctas);
  p.teams = a->num_ctas / p.team;
  p.cut = static_cast<int4*>(a->workspace);
  p.ws_o = reinterpret_cast<float*>(static_cast<char*>(a->workspace) + o_at);
  p.ws_l = reinterpret_cast<float*>(static_cast<char*>(a->workspace) + l_at);
  p.status = a->status_dev;
  p.timeout_ns = attn_debug().timeout_ns;
  p.withhold_q = attn_debug().withhold_q;
  TreeMaps m;
  auto map = [&](CUtensorMap* t, const void* base, int64_t hs, int64_t rs, int box_rows) {
    return make_rows_map(t, base, d, quant, Hkv, a->num_kv_rows, hs, rs, box_rows);
  };
  const int whole = std::min(BN, page);
  if (!map(&m.k, a->k, a->k_head_stride, a->k_row_stride, whole) ||
      !map(&m.v, a->v, a->v_head_stride, a->v_row_stride, whole))
    return CPATTN_ERR_CUDA;
  if (whole > 16) {
    if (!map(&m.k_tail, a->k, a->k_head_stride, a->k_row_stride, 16) ||
        !map(&m.v_tail, a->v, a->v_head_stride, a->v_row_stride, 16))
      return CPATTN_ERR_CUDA;
  } else {
    m.k_tail = m.k;
    m.v_tail = m.v;
  }
  // (a map wants strides; the slow way takes any)
  p.q_boxes = !quant && p.unit_rows >= BM && BM % p.g == 0 && p.q_row > 0 && p.q_head > 0 &&
              make_q_map(&m.q, a->q, d, a->Hq, a->num_rows, p.q_head, p.q_row, p.g);
  const int r = p.unit_rows < BM ? launch_tree_small(m, p, d, quant, a->num_ctas, stream)
                                 : launch_tree_mma(m, p, d, quant, a->num_ctas, stream);
  if (r != CPATTN_OK) return r;
  return (d == 128 ? launch_merge<128>(p, a->num_ctas, stream) : launch_merge<64>(p, a->num_ctas, stream)) ==
                 cudaSuccess
             ? CPATTN_OK
             : CPATTN_ERR_CUDA;
}
