// Attention over a paged cache (cp_attn_tree): its work list and launch parameters.
//
// A unit is a KV head of a request and up to `unit_rows` of its packed rows (new row i, head
// j of the KV head's group, at i*g + j).  The units' KV tiles of 128 keys, by request, head,
// row tile and key, form one line, which is cut into equal shares, one a thread block.  The
// blocks find their shares themselves, from the lengths on the device: a scan over the requests
// in each block, then a walk.  So a launch depends on no length, and a captured graph serves
// every step.
//
// A unit inside one share is finished by its block.  One that is cut leaves a partial (O, L)
// in the workspace for each of its blocks: a block has at most two, its first piece (slot 2c,
// when the unit began in an earlier block) and its last (slot 2c + 1, when it began here and
// goes on).  The block where a cut unit begins describes it for the merge.
#pragma once
#include <cstdint>

#include "attn_tiles.cuh"

namespace cpattn {

struct TreeParams {
  const int32_t *q_start, *kv_lens, *page_table, *mask;
  long long table_stride;
  int num_reqs, num_rows, max_pages, log_page, words;
  int Hq, Hkv, g;
  uint32_t g_mul, g_shift;  // see group_div
  int unit_rows;
  const __nv_bfloat16* q;
  long long q_row, q_head;
  const float *ks, *vs;
  long long s_head;
  int num_kv_rows;
  float scale_log2;
  void* o;
  int o_f32;
  float* lse;
  float* ws_o;  // [slots][dv / 8][unit_rows][8]
  float* ws_l;  // [slots][unit_rows], log2 units
  int4* cut;    // [num_ctas][2]: the unit that is cut behind this block, see TreeCut
  int32_t* status;
  unsigned long long timeout_ns;
  int withhold_q;  // test hook: queries are never published (see cp_attn_debug)
};

// A cut unit: first query row of its request, first packed row, rows, KV head; blocks (0: none).
struct TreeCut {
  int row0, r0, rows, kv_head, blocks;
};

// The kernel for up to `unit_rows` rows a unit on warp-level MMAs (attn_tree_small.cu):
// 8, 16 or 32 rows; pages: boxes of whole pages (at most 128 rows) and of 16 rows.
struct TreeMaps {
  CUtensorMap k, v, k_tail, v_tail;
};
// Whether a launch of `kern` has the registers that its warps share out (setmaxnreg.inc waits
// for them): a property of this binary.
template <typename... Params>
inline bool split_covered(void (*kern)(Params...), int threads, int regs) {
  cudaFuncAttributes fa;
  return cudaFuncGetAttributes(&fa, kern) == cudaSuccess && fa.numRegs * threads >= regs;
}
int launch_tree_small(const TreeMaps& m, const TreeParams& p, int d, bool quant, int num_ctas, cudaStream_t stream);
// ... and the one on tcgen05 (attn_tree_mma.cu): 128 or 256 rows.
int launch_tree_mma(const TreeMaps& m, const TreeParams& p, int d, bool quant, int num_ctas, cudaStream_t stream);

namespace {

struct TreeReq {
  int row0, T, L;  // first query row, new rows, cached keys
};
__device__ __forceinline__ TreeReq load_req(const TreeParams& p, int b, bool& bad) {
  const int s0 = __ldg(p.q_start + b), s1 = __ldg(p.q_start + b + 1), L = __ldg(p.kv_lens + b);
  const long long T = (long long)s1 - s0, keys = L + T;
  bad = s0 < 0 || T < 0 || s1 > p.num_rows || (b == 0 && s0 != 0) ||
        (T > 0 && (L < 0 || keys > (long long)p.max_pages << p.log_page || keys > 0x7fffffffLL - 2 * BN ||
                   (p.mask && T > 32LL * p.words)));
  return bad ? TreeReq{0, 0, 0} : TreeReq{s0, (int)T, L};
}
__device__ __forceinline__ int row_tiles(const TreeParams& p, const TreeReq& r) {
  return (int)(((long long)r.T * p.g + p.unit_rows - 1) / p.unit_rows);
}
__device__ __forceinline__ long long req_cost(const TreeParams& p, const TreeReq& r) {
  return r.T == 0 ? 0 : (long long)row_tiles(p, r) * p.Hkv * num_tiles(r.L + r.T);
}

// Where a block's share begins.
struct TreeStart {
  long long at, end, b0;  // the share, and the place of request b's first tile
  long long share;
  int b;
};

// All threads of the block; sums: a word for each warp.
__device__ __forceinline__ TreeStart tree_start(const TreeParams& p, long long* sums, long long* found) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int per = (p.num_reqs + blockDim.x - 1) / blockDim.x;
  const long long lo = (long long)threadIdx.x * per, hi = min((long long)p.num_reqs, lo + per);
  long long sum = 0;
  bool any = false;
  for (long long b = lo; b < hi; ++b) {
    bool bad;
    sum += req_cost(p, load_req(p, (int)b, bad));
    any = any || bad;
  }
  if (any) set_status(p.status, CPATTN_ERR_RANGE);
  long long upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  long long total = 0, before = 0;
  for (int w = 0; w < warps; ++w) {
    if (w == warp) before = total;
    total += sums[w];
  }
  TreeStart s;
  s.share = max(1LL, (total + gridDim.x - 1) / gridDim.x);
  s.at = s.share * blockIdx.x;
  s.end = min(total, s.at + s.share);
  before += upto - sum;
  if (s.at >= before && s.at < before + sum)
    for (long long b = lo; b < hi; ++b) {
      bool bad;
      const long long cost = req_cost(p, load_req(p, (int)b, bad));
      if (s.at < before + cost) {
        found[0] = b;
        found[1] = before;
        break;
      }
      before += cost;
    }
  __syncthreads();
  s.b = s.at < s.end ? (int)found[0] : 0;
  s.b0 = s.at < s.end ? found[1] : 0;
  return s;
}

struct TreePiece {
  TreeReq req;
  int b, kv_head;
  int r0, rows;    // first packed row of the unit and its rows
  int t0, tiles;   // KV tiles
  int keys;        // of the unit
  int slot;        // of the partial, -1: the unit is whole
  int blocks;      // that the unit is cut over, when it begins here and is cut; else 0
};

// Steps through a share; every role of a block walks on its own.
struct TreeWalk {
  TreeStart s;
  __device__ __forceinline__ bool next(const TreeParams& p, TreePiece& pc) {
    while (s.at < s.end) {
      bool bad;
      const TreeReq r = load_req(p, s.b, bad);
      const int tiles = num_tiles(max(1, r.L + r.T)), rts = row_tiles(p, r);
      const long long cost = r.T == 0 ? 0 : (long long)rts * p.Hkv * tiles;
      if (s.at >= s.b0 + cost) {
        s.b0 += cost;
        ++s.b;
        continue;
      }
      const long long unit = (s.at - s.b0) / tiles, w0 = s.b0 + unit * tiles;
      const int t0 = (int)(s.at - w0), t1 = (int)min((long long)tiles, s.end - w0);
      s.at = w0 + t1;
      pc.req = r;
      pc.b = s.b;
      pc.kv_head = (int)(unit / rts);
      pc.r0 = (int)(unit - (long long)pc.kv_head * rts) * p.unit_rows;
      pc.rows = (int)min((long long)p.unit_rows, (long long)r.T * p.g - pc.r0);
      pc.keys = p.mask ? r.L + r.T : r.L + group_div(p, pc.r0 + pc.rows - 1) + 1;
      const int nt = num_tiles(pc.keys);
      pc.t0 = t0;
      pc.tiles = min(nt, t1) - t0;
      if (pc.tiles <= 0) continue;  // (keys that only the request's later rows see)
      const long long c0 = w0 / s.share, c1 = (w0 + nt - 1) / s.share;
      pc.slot = c0 == c1 ? -1 : 2 * (int)blockIdx.x + (c0 == blockIdx.x ? 1 : 0);
      pc.blocks = c0 == blockIdx.x && c1 > c0 ? (int)(c1 - c0) + 1 : 0;
      return true;
    }
    return false;
  }
};

__device__ __forceinline__ void put_cut(const TreeParams& p, const TreePiece& pc, int blocks) {
  p.cut[2 * blockIdx.x] = make_int4(pc.req.row0, pc.r0, pc.rows, pc.kv_head);
  p.cut[2 * blockIdx.x + 1] = make_int4(blocks, 0, 0, 0);
}

// Cache row of key `key` of request b (key within the request's pages).  A page outside the
// cache gives a row behind it, which the TMA reads as zeros.
__device__ __forceinline__ int cache_row(const TreeParams& p, int b, int key) {
  const int page = __ldg(p.page_table + b * p.table_stride + (key >> p.log_page));
  if ((uint32_t)page >= (uint32_t)(p.num_kv_rows >> p.log_page)) {
    set_status(p.status, CPATTN_ERR_RANGE);
    return p.num_kv_rows;
  }
  return (page << p.log_page) + (key & ((1 << p.log_page) - 1));
}

// Whether new row `node` of a request sees new key `n` (0 <= n < T).
__device__ __forceinline__ bool sees(const TreeParams& p, const TreeReq& r, int node, int n) {
  if (!p.mask) return n <= node;
  return ((uint32_t)__ldg(p.mask + (long long)(r.row0 + node) * p.words + (n >> 5)) >> (n & 31)) & 1u;
}

}  // namespace
}  // namespace cpattn
