// Attention over a paged cache (cp_attn_tree): its work list and launch parameters.
//
// A unit is a KV head of a request and up to `unit_rows` of its packed rows (new row i, head
// j of the KV head's group, at i*g + j).  A team of blocks takes one unit each of as many KV
// heads that lie side by side, and walks the same keys: a cache row holds all heads' parts, and
// so what DRAM opens for one head is read for the others while it is open.  The units' KV tiles
// of 128 keys, by request, heads, row tile and key, form one line, which is cut into equal
// shares, one a team.  The blocks find their shares themselves, from the lengths on the
// device: a scan over the requests in each block, then a walk.  So a launch depends on no
// length, and a captured graph serves every step.
//
// A unit inside one share is finished by its block.  One that is cut leaves a partial (O, L)
// in the workspace for each of its blocks, c, c + team, ...: a block has at most two, its first
// piece (slot 2c, when the unit began in an earlier share) and its last (slot 2c + 1, when it
// began here and goes on).  The block where a cut unit begins describes it for the merge.
#pragma once
#include <atomic>
#include <cstdint>

#include "attn_tiles.cuh"

namespace cpattn {

struct TreeParams {
  const int32_t *q_start, *kv_lens, *page_table, *mask;
  long long table_stride;
  int num_reqs, num_rows, max_pages, log_page, words;
  int Hq, Hkv, g;
  uint32_t g_mul, g_shift;  // see group_div
  int unit_rows, unit_log;  // 2^unit_log
  int team, teams;  // blocks of a team, teams
  const __nv_bfloat16* q;
  long long q_row, q_head;
  const float *ks, *vs;
  long long s_head;
  int scales_16;  // 16 keys' scales begin at 16-byte boundaries
  int num_kv_rows;
  float scale_log2;
  void* o;
  int o_f32, o_32;  // fp32; 32-byte aligned
  int q_boxes;      // a tile's 128 packed rows are a box of the queries: all heads of 128 / g rows
  float* lse;
  float* ws_o;  // [slots][dv / 8][unit_rows][8]
  float* ws_l;  // [slots][unit_rows], log2 units
  // [num_ctas][2]: of the unit that is cut behind this block the request's first query row, the first
  // packed row, the rows and the KV head; the blocks (0: none is cut)
  int4* cut;
  int32_t* status;
  unsigned long long timeout_ns;
  int withhold_q;  // test hook: queries are never published (see cp_attn_debug)
};

// Pages come as boxes of whole pages (at most 128 rows), a unit's end as boxes of 16 rows.
struct TreeMaps {
  CUtensorMap k, v, k_tail, v_tail;
  CUtensorMap q;  // with TreeParams::q_boxes
};
// Whether a launch of `kern` has the registers that its warps share out (setmaxnreg.inc waits
// for them): a property of this binary, kept in `known` (0: not asked, 1: yes, -1: no).
template <typename... Params>
inline bool split_covered(void (*kern)(Params...), int threads, int regs, std::atomic<int>& known) {
  int k = known.load(std::memory_order_relaxed);
  if (k == 0) {
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return false;
    k = fa.numRegs * threads >= regs ? 1 : -1;
    known.store(k, std::memory_order_relaxed);
  }
  return k > 0;
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
  return (int)(((long long)r.T * p.g + p.unit_rows - 1) >> p.unit_log);
}
__device__ __forceinline__ long long req_cost(const TreeParams& p, const TreeReq& r) {
  return r.T == 0 ? 0 : (long long)row_tiles(p, r) * (p.Hkv / p.team) * num_tiles(r.L + r.T);
}

// Where a block's share begins.
struct TreeStart {
  long long first, at, end, b0;  // the share, and the place of request b's first tile
  long long share;
  int b;
};

// All threads of the block, of WARPS warps; sums: a word for each, in shared memory as found's two.
template <int WARPS>
__device__ __forceinline__ TreeStart tree_start(const TreeParams& p, long long (&sums)[WARPS], long long* found) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
  for (int w = 0; w < WARPS; ++w) {
    if (w == warp) before = total;
    total += sums[w];
  }
  TreeStart s;
  s.share = max(1LL, (total + p.teams - 1) / p.teams);
  s.first = s.share * (blockIdx.x / p.team);
  s.at = s.first;
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
  int row0, T, L, b;       // the request
  int kv_head, r0, rows;   // first packed row of the unit and its rows
  int t0, tiles, keys;     // KV tiles of the piece (0: there is none), keys of the unit
  int slot;                // of the partial, -1: the unit is whole
  int blocks;              // that the unit is cut over, when it begins here and is cut; else 0
};
static_assert(sizeof(TreePiece) == 48, "three 16-byte words");

// Steps through a share.  The next request's words are loaded while the one at hand is walked:
// under load they are a few thousand cycles away.
struct TreeWalk {
  TreeStart s;
  TreeReq r, ahead;
  long long w0;  // place of the unit at hand
  int tiles, rts, heads, rt;  // heads: of the team, their number
  __device__ __forceinline__ TreeReq load(const TreeParams& p, int b) const {
    bool bad;
    return b < p.num_reqs ? load_req(p, b, bad) : TreeReq{0, 0, 0};
  }
  __device__ __forceinline__ void take(const TreeParams& p) {
    tiles = num_tiles(max(1, r.L + r.T));
    rts = row_tiles(p, r);
  }
  __device__ __forceinline__ TreeWalk(const TreeParams& p, const TreeStart& start) : s(start) {
    tiles = rts = 1;
    heads = rt = 0;
    w0 = 0;
    if (s.at >= s.end) return;
    r = load(p, s.b);
    ahead = load(p, s.b + 1);
    take(p);
    const long long unit = (s.at - s.b0) / tiles;
    w0 = s.b0 + unit * tiles;
    heads = (int)(unit / rts);
    rt = (int)(unit - (long long)heads * rts);
  }
  __device__ __forceinline__ bool next(const TreeParams& p, TreePiece& pc) {
    while (s.at < s.end) {
      pc.row0 = r.row0;
      pc.T = r.T;
      pc.L = r.L;
      pc.b = s.b;
      pc.kv_head = heads * p.team + (int)blockIdx.x % p.team;
      pc.r0 = rt * p.unit_rows;
      pc.rows = (int)min((long long)p.unit_rows, (long long)r.T * p.g - pc.r0);
      pc.keys = p.mask ? r.L + r.T : r.L + group_div(p, pc.r0 + pc.rows - 1) + 1;
      const int nt = num_tiles(pc.keys);
      pc.t0 = (int)(s.at - w0);
      pc.tiles = (int)min((long long)nt, s.end - w0) - pc.t0;
      const bool here = w0 >= s.first, cut = w0 + nt > s.end;
      pc.slot = here && !cut ? -1 : 2 * (int)blockIdx.x + (here ? 1 : 0);
      pc.blocks = here && cut ? (int)((w0 + nt - 1) / s.share - s.first / s.share) + 1 : 0;
      // on to the next unit
      s.at = min(s.end, w0 + tiles);
      w0 += tiles;
      if (++rt == rts) {
        rt = 0;
        if (++heads == p.Hkv / p.team && s.at < s.end) {
          heads = 0;
          do {
            ++s.b;
            r = ahead;
            ahead = load(p, s.b + 1);
          } while (r.T == 0 && s.b < p.num_reqs);
          take(p);
        }
      }
      if (pc.tiles > 0) return true;  // (else keys that only the request's later rows see)
    }
    return false;
  }
};

// The block's pieces, walked by one warp and read by the others; the last has no tiles.
template <int N>
struct PieceRing {
  TreePiece at[N];
  uint64_t full[N], empty[N];
  __device__ __forceinline__ void init(int readers) {
    for (int i = 0; i < N; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, readers);
    }
  }
  // Piece i, by a whole warp; false when a wait ran out.
  __device__ __forceinline__ bool put(int i, const TreePiece& pc, const volatile int* abort, uint64_t timeout) {
    if (!wait_warp(empty + i % N, ((i / N) & 1) ^ 1, abort, timeout)) return false;
    if ((threadIdx.x & 31) == 0) {
      at[i % N] = pc;
      mbar_arrive(full + i % N);
    }
    return true;
  }
  // ... read; without tiles when there is none or a wait ran out.
  __device__ __forceinline__ bool get(int i, TreePiece& pc, const volatile int* abort, uint64_t timeout) {
    pc.tiles = 0;
    if (!wait_warp(full + i % N, (i / N) & 1, abort, timeout)) return false;
    const int4* w = reinterpret_cast<const int4*>(at + i % N);
    const int4 a = w[0], b = w[1], c = w[2];
    pc = TreePiece{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
    return true;
  }
  // A reader is done with piece i (one of a warp).
  __device__ __forceinline__ void done(int i) { mbar_arrive(empty + i % N); }
};

__device__ __forceinline__ void put_cut(const TreeParams& p, const TreePiece& pc, int blocks) {
  p.cut[2 * blockIdx.x] = make_int4(pc.row0, pc.r0, pc.rows, pc.kv_head);
  p.cut[2 * blockIdx.x + 1] = make_int4(blocks, 0, 0, 0);
}

// The warp that walks the share puts its pieces into the ring, and reads them there itself.
template <int N>
struct TreeWalker {
  TreeWalk w;
  PieceRing<N>& ring;
  int walked = 0;
  bool more = true, ok = true, cut = false;
  __device__ __forceinline__ TreeWalker(const TreeParams& p, const TreeStart& start, PieceRing<N>& r)
      : w(p, start), ring(r) {}
  // Pieces up to number n, and the one without tiles behind the last.
  __device__ __forceinline__ void upto(const TreeParams& p, int n, const volatile int* abort) {
    for (; more && ok && walked <= n; ++walked) {
      TreePiece x;
      more = w.next(p, x);
      if (!more) x.tiles = x.rows = x.blocks = 0;
      if (x.blocks) {
        cut = true;
        if ((threadIdx.x & 31) == 0) put_cut(p, x, x.blocks);
      }
      ok = ring.put(walked, x, abort, p.timeout_ns);
    }
  }
  // By one lane, when there are no more.
  __device__ __forceinline__ void end(const TreeParams& p) const {
    if (!cut) p.cut[2 * blockIdx.x + 1] = make_int4(0, 0, 0, 0);
  }
};

// A KV tile for its loader.  The lane's box is whole pages, or 16 rows of a unit's end.
struct LoadTile {
  int live;          // keys of the unit from the tile's first on, at most BN; 0: no tile
  int log;           // rows of a box (log2)
  int page, at;      // of the lane's box: entry of the page table, row in the page
  int kv_head, fresh, t;  // fresh: the first row that is a new key; t: number in the piece
  // Cache row of the lane's box; of a page outside the cache a row behind it, which TMA reads
  // as zeros.
  __device__ __forceinline__ int row(const TreeParams& p) const {
    return (uint32_t)page < (uint32_t)(p.num_kv_rows >> p.log_page) ? (page << p.log_page) + at : p.num_kv_rows;
  }
};
// The KV tiles of the block's pieces.  A loader takes a tile ahead of the one that it copies,
// and looks at its page table's words only then: under load they are a thousand cycles away
// (e4m3 tiles of 16-row pages: 142 -> 123 us a decode step of 64).
template <int N>
struct TileLoader {
  PieceRing<N>& ring;
  TreePiece pc;
  int i = -1, t = 0;  // piece, its tile
  bool ok = true, end = false;
  __device__ __forceinline__ explicit TileLoader(PieceRing<N>& r) : ring(r) { pc.tiles = 0; }
  __device__ __forceinline__ LoadTile next(const TreeParams& p, const volatile int* abort) {
    LoadTile x;
    x.live = x.log = x.page = x.at = x.kv_head = x.fresh = x.t = 0;
    if (end) return x;
    if (++t >= pc.tiles) {
      ok = ring.get(++i, pc, abort, p.timeout_ns);
      end = pc.tiles == 0;
      if (end) return x;
      t = 0;
    }
    const int key0 = (pc.t0 + t) * BN, mine = threadIdx.x & 31;
    x.live = min(BN, pc.keys - key0);
    x.log = x.live > BN - 16 ? min(7, p.log_page) : 4;
    const int key = key0 + (mine << x.log);
    if ((mine << x.log) < x.live) x.page = __ldg(p.page_table + pc.b * p.table_stride + (key >> p.log_page));
    x.at = key & ((1 << p.log_page) - 1);
    x.kv_head = pc.kv_head;
    x.fresh = pc.L - key0;
    x.t = t;
    return x;
  }
};
// Starts the copies of a tile, kChunks boxes of 64 columns across, by the lanes that hold the
// rows (one lane that starts them all takes 2900 cycles for 8 pages, these 2200).
template <int kChunks, int kLine>
__device__ __forceinline__ void copy_tile(const TreeParams& p, const CUtensorMap* whole, const CUtensorMap* tail,
                                          uint8_t* dst, uint64_t* bar, const LoadTile& x, int row, int whole_log) {
  const int lane = threadIdx.x & 31, boxes = (x.live + (1 << x.log) - 1) >> x.log;
  if (lane == 0) mbar_arrive_expect_tx(bar, (boxes << x.log) * kLine * kChunks);
  __syncwarp();
  if (lane < boxes) {
    const CUtensorMap* tm = x.log == whole_log ? whole : tail;
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
      tma_load_3d(dst + (c * BN + (lane << x.log)) * kLine, tm, bar, c * 64, x.kv_head, row);
    if (row == p.num_kv_rows) set_status(p.status, CPATTN_ERR_RANGE);
  }
  __syncwarp();
}
// The scales of a tile's rows to `at` in shared memory, asynchronously: whole blocks of 16 keys,
// which lie in a page, or a word a key where their addresses are not aligned.
__device__ __forceinline__ void copy_scales(const TreeParams& p, const float* scales, const LoadTile& x, int row,
                                            uint32_t at) {
  const int lane = threadIdx.x & 31;
  const float* from = scales + (long long)x.kv_head * p.s_head;
  if (p.scales_16) {
    const int key = 16 * (lane >> 2), r = __shfl_sync(0xffffffffu, row, key >> x.log) + (key & ((1 << x.log) - 1));
    if (key < x.live && r < p.num_kv_rows)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at + lane * 16), "l"(from + r + 4 * (lane & 3))
                   : "memory");
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int key = i * 32 + lane, r = __shfl_sync(0xffffffffu, row, key >> x.log) + (key & ((1 << x.log) - 1));
    if (key < x.live && r < p.num_kv_rows)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(at + key * 4), "l"(from + r) : "memory");
  }
}
// Arrives when this lane's copies so far have landed.
__device__ __forceinline__ void arrive_copies(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Ring place of K and V of a list's n-th KV tile, in the order of use: K0 V0 K1 V1 ..., or
// (AHEAD: two streams take turns) K0 K1 V0 K2 V1 ..., where the place behind the last V but
// one is left out.
template <bool AHEAD>
__device__ __forceinline__ int k_place(int n) { return !AHEAD ? 2 * n : n == 0 ? 0 : 2 * n - 1; }
template <bool AHEAD>
__device__ __forceinline__ int v_place(int n) { return !AHEAD ? 2 * n + 1 : 2 * n + 2; }
// Waits for the copies in flight, of nk K and nv V tiles, after an abort: the last of each slot.
template <bool AHEAD>
__device__ __forceinline__ void drain_tiles(uint64_t* full, int stages, int nk, int nv, uint64_t timeout) {
  for (int slot = 0; slot < stages; ++slot) {
    int last = -1;
    for (int n = max(0, nk - stages - 1); n < nk; ++n)
      if (k_place<AHEAD>(n) % stages == slot) last = max(last, k_place<AHEAD>(n));
    for (int n = max(0, nv - stages - 1); n < nv; ++n)
      if (v_place<AHEAD>(n) % stages == slot) last = max(last, v_place<AHEAD>(n));
    if (last >= 0) wait_one(full + slot, (last / stages) & 1, nullptr, timeout);
  }
}

// Whether new row `node` of a request sees new key `n` (0 <= n < T).
__device__ __forceinline__ bool sees(const TreeParams& p, const TreePiece& pc, int node, int n) {
  if (!p.mask) return n <= node;
  return ((uint32_t)__ldg(p.mask + (long long)(pc.row0 + node) * p.words + (n >> 5)) >> (n & 31)) & 1u;
}

// Brings the masks of a piece's rows to L1, by a whole warp (up to 8 KB).
__device__ __forceinline__ void fetch_masks(const TreeParams& p, const TreePiece& pc) {
  if (!p.mask) return;
  const int n0 = group_div(p, pc.r0), n1 = group_div(p, pc.r0 + pc.rows - 1);
  const char* at = reinterpret_cast<const char*>(p.mask + (long long)(pc.row0 + n0) * p.words);
  const long long bytes = min(8192LL, (long long)(n1 - n0 + 1) * p.words * 4);
  for (long long x = (threadIdx.x & 31) * 32; x < bytes; x += 32 * 32)
    asm volatile("prefetch.global.L1 [%0];" ::"l"(at + x));
}

}  // namespace
}  // namespace cpattn
