// Layout of a decode step over a paged cache (cp_tree_layout): where the new rows go,
// their positions, and each node's ancestors as bits.
//
// A node's ancestors have lower numbers, so that a walk from the node to its root meets
// falling bits: a thread a node keeps the current word in a register and writes each word
// once.  A block a request, the parents in shared memory.  Latency: the walk is as long as
// the node is deep, each step a shared-memory load (4.5 us for 256 requests of up to 64
// nodes, 2.1 for one of 8, the launch among them).
#include <algorithm>
#include <cstdint>

#include "../../include/cpattn.h"
#include "ptx.cuh"
#include "trace.h"

namespace cpattn {
namespace {

constexpr int kThreads = 64;
constexpr int kHeld = 2048;  // parents in shared memory; those of longer requests are read where they are

struct LayoutParams {
  const int32_t* q_start;
  const int32_t* kv_lens;
  const int32_t* page_table;
  long long table_stride;
  const int32_t* parents;
  int32_t *slots, *positions, *mask, *status;
  int num_reqs, max_pages, log_page, num_rows, words;
};

__global__ void __launch_bounds__(kThreads) tree_layout_kernel(const LayoutParams p) {
  __shared__ int32_t held[kHeld];
  const int b = blockIdx.x;
  auto none = [&](long long row) {  // a row of no request
    p.slots[row] = -1;
    p.positions[row] = 0;
    if (p.mask)
      for (int w = 0; w < p.words; ++w) p.mask[row * p.words + w] = 0;
  };
  if (b >= p.num_reqs) {  // padding rows
    const int first = max(0, p.num_reqs > 0 ? __ldg(p.q_start + p.num_reqs) : 0);
    for (long long row = first + (long long)(b - p.num_reqs) * kThreads + threadIdx.x; row < p.num_rows;
         row += (long long)(gridDim.x - p.num_reqs) * kThreads)
      none(row);
    return;
  }
  const int s0 = __ldg(p.q_start + b), s1 = __ldg(p.q_start + b + 1), len = __ldg(p.kv_lens + b);
  if (s0 < 0 || s1 < s0 || s1 > p.num_rows || (b == 0 && s0 != 0)) {
    if (threadIdx.x == 0) set_status(p.status, CPATTN_ERR_RANGE);
    // the rows between its ends, which may be no other's: an append that follows must not find
    // there what the memory held (from row 0 on to the end of q_start each row is between some two)
    const int hi = min(p.num_rows, max(s0, s1));
    for (long long row = (b == 0 ? 0 : max(0, min(s0, s1))) + (long long)threadIdx.x; row < hi; row += kThreads) none(row);
    return;
  }
  const int T = s1 - s0;
  const bool fits = len >= 0 && (long long)len + T <= (long long)p.max_pages << p.log_page &&
                    (long long)len + T <= 0x7fffffffLL;
  if (!fits && T > 0 && threadIdx.x == 0) set_status(p.status, CPATTN_ERR_RANGE);
  const int32_t* up = p.parents ? p.parents + s0 : nullptr;
  if (up && T <= kHeld) {
    for (int i = threadIdx.x; i < T; i += kThreads) held[i] = __ldg(up + i);
    up = held;
    __syncthreads();
  }
  for (int i = threadIdx.x; i < T; i += kThreads) {
    const long long row = (long long)s0 + i;
    int slot = -1;
    if (fits) {
      const int at = len + i, page = __ldg(p.page_table + b * p.table_stride + (at >> p.log_page));
      const long long to = ((long long)page << p.log_page) + (at & ((1 << p.log_page) - 1));
      if (page >= 0 && to <= 0x7fffffffLL) slot = (int)to;
      else set_status(p.status, CPATTN_ERR_RANGE);
    }
    int depth = i;
    if (up) {
      depth = 0;
      int word = p.words - 1;  // the word that is being gathered; those above it are written
      uint32_t bits = 0;
      bool ok = i < 32LL * p.words;
      for (int j = i;;) {
        if (p.mask && (j >> 5) < p.words) {
          for (; word > (j >> 5); --word, bits = 0) p.mask[row * p.words + word] = (int32_t)bits;
          bits |= 1u << (j & 31);
        }
        const int next = up[j];
        if (next < 0 || next >= j) {
          ok = ok && next == -1;
          break;
        }
        j = next;
        ++depth;
      }
      if (p.mask)
        for (; word >= 0; --word, bits = 0) p.mask[row * p.words + word] = (int32_t)bits;
      if (!ok) set_status(p.status, CPATTN_ERR_RANGE);
    }
    p.slots[row] = slot;
    p.positions[row] = fits ? len + depth : 0;
  }
}

}  // namespace
}  // namespace cpattn

using namespace cpattn;

extern "C" int cp_tree_layout(const cp_tree_layout_args_t* a, cudaStream_t stream) {
  CPATTN_TRACE("cp_tree_layout");
  if (!a) return CPATTN_ERR_INVALID_ARG;
  if (a->num_reqs < 0 || a->num_reqs > CPATTN_MAX_REQS || a->num_rows < 0 || a->max_pages < 0 || a->mask_words < 0 ||
      (a->parents != nullptr) != (a->mask != nullptr && a->mask_words > 0) || (a->mask && !a->parents))
    return CPATTN_ERR_INVALID_ARG;
  if (a->page_size < 16 || a->page_size > 65536 || (a->page_size & (a->page_size - 1))) return CPATTN_ERR_UNSUPPORTED;
  if (a->num_reqs > 1 && a->table_stride < a->max_pages) return CPATTN_ERR_INVALID_ARG;
  for (const void* at : {(const void*)a->q_start, (const void*)a->kv_lens, (const void*)a->page_table,
                         (const void*)a->parents, (const void*)a->slots, (const void*)a->positions,
                         (const void*)a->mask, (const void*)a->status_dev})
    if (reinterpret_cast<uintptr_t>(at) & 3u) return CPATTN_ERR_ALIGNMENT;
  if (a->num_rows == 0) return CPATTN_OK;
  if (!a->slots || !a->positions ||
      (a->num_reqs > 0 && (!a->q_start || !a->kv_lens || (a->max_pages > 0 && !a->page_table))))
    return CPATTN_ERR_INVALID_ARG;
  LayoutParams p{};
  p.q_start = a->q_start;
  p.kv_lens = a->kv_lens;
  p.page_table = a->page_table;
  p.table_stride = a->table_stride;
  p.parents = a->parents;
  p.slots = a->slots;
  p.positions = a->positions;
  p.mask = a->mask;
  p.status = a->status_dev;
  p.num_reqs = a->num_reqs;
  p.max_pages = a->max_pages;
  for (p.log_page = 4; (1 << p.log_page) < a->page_size; ++p.log_page) {}
  p.num_rows = a->num_rows;
  p.words = a->mask_words;
  const unsigned pad = (unsigned)std::min<long long>(((long long)a->num_rows + kThreads - 1) / kThreads, 32);
  tree_layout_kernel<<<a->num_reqs + pad, kThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? CPATTN_OK : CPATTN_ERR_CUDA;
}
