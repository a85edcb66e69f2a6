// What the operators on the paged key/value cache share: the element types,
// the address of a cache slot, and the check of one request's data.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "specverify.h"

namespace specv_cache_ops {

constexpr int kMaxNodes = SPECV_MAX_NODES;
constexpr int kSms = 152;  // of a GB300: what the rules for splits and variants were measured on
constexpr unsigned kFullMask = 0xffffffffu;

struct Bf16 {
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};

struct F16 {
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};

// The cache as the kernels take it (specv_cache, with 16-bit elements).
struct Cache {
  uint16_t* k;
  uint16_t* v;
  const int32_t* page_table;
  const int32_t* lens;
  int64_t layer_stride, page_stride, row_stride, head_stride;
  int layers, pages, page_size, max_pages, table_stride, heads, head_dim;

  // Offset of request b's slot s in elements.  Its page number was checked.
  __device__ __forceinline__ int64_t slot(int b, int s) const {
    const int page = s / page_size;
    return static_cast<int64_t>(page_table[static_cast<int64_t>(b) * table_stride + page]) *
               page_stride +
           static_cast<int64_t>(s - page * page_size) * row_stride;
  }
};

struct Rows {
  uint16_t* data;
  int64_t batch_stride, node_stride, head_stride;
};

// One request's tree, as a warp holds it: lane l has nodes l and l + 32.
struct Tree {
  int n;         // nodes, 0 if the count itself is bad
  int len;       // verified tokens in the cache
  unsigned bad;  // SPECV_DEV_* bits
  int up[2];     // parent of this lane's nodes; -1 at the root and behind the last
};

__device__ __forceinline__ int at_node(const int (&x)[2], int i) {
  const int lo = __shfl_sync(kFullMask, x[0], i & 31);
  const int hi = __shfl_sync(kFullMask, x[1], i & 31);
  return i < 32 ? lo : hi;
}

// Reads the node count, the length and the parents of request b and checks
// them (every lane of a warp calls this; bad is the same on every lane).
__device__ __forceinline__ Tree read_tree(const int32_t* parents, const int32_t* n_nodes,
                                          const int32_t* lens, int b, int N, int64_t slots,
                                          int lane) {
  Tree t;
  t.n = n_nodes ? n_nodes[b] : N;
  t.len = lens[b];
  int up[2] = {-1, -1};
#pragma unroll
  for (int k = 0; k < 2; k++) {
    const int i = lane + 32 * k;
    if (i < N) up[k] = parents ? parents[static_cast<int64_t>(b) * N + i] : i - 1;
  }
  t.bad = 0;
  if (t.n < 1 || t.n > N) {
    t.bad |= SPECV_DEV_BAD_DRAFT_LEN;
    t.n = 0;
  }
  if (t.len < 0 || t.len > INT_MAX - 4 * kMaxNodes ||
      static_cast<int64_t>(t.len) + t.n > slots)
    t.bad |= SPECV_DEV_BAD_CACHE;
  bool bad_tree = false;
#pragma unroll
  for (int k = 0; k < 2; k++) {
    const int i = lane + 32 * k;
    if (i < t.n) bad_tree |= i == 0 ? up[k] != -1 : up[k] < 0 || up[k] >= i;
    t.up[k] = i < t.n ? up[k] : -1;
  }
  if (__any_sync(kFullMask, bad_tree)) t.bad |= SPECV_DEV_BAD_TREE;
  return t;
}

// Depth of this lane's nodes by pointer doubling: after r rounds a node knows
// its distance to the ancestor 2^r above it, so six rounds reach 64 nodes.
// Only for a tree that read_tree found good.
__device__ __forceinline__ void depths(const Tree& t, int (&depth)[2]) {
  int up[2] = {t.up[0], t.up[1]};
  depth[0] = up[0] >= 0;
  depth[1] = up[1] >= 0;
#pragma unroll
  for (int r = 0; r < 6; r++) {
    int d[2], u[2];
#pragma unroll
    for (int k = 0; k < 2; k++) {
      d[k] = at_node(depth, up[k] & 63);
      u[k] = at_node(up, up[k] & 63);
    }
#pragma unroll
    for (int k = 0; k < 2; k++)
      if (up[k] >= 0) {
        depth[k] += d[k];
        up[k] = u[k];
      }
  }
}

// Bit j of a node's word: j is the node or one of its ancestors.
__device__ __forceinline__ void ancestors(const Tree& t, int lane, uint64_t (&bits)[2]) {
  int up[2] = {t.up[0], t.up[1]};
  int lo[2] = {static_cast<int>(1u << lane), 0}, hi[2] = {0, static_cast<int>(1u << lane)};
#pragma unroll
  for (int r = 0; r < 6; r++) {
    int l[2], h[2], u[2];
#pragma unroll
    for (int k = 0; k < 2; k++) {
      l[k] = at_node(lo, up[k] & 63);
      h[k] = at_node(hi, up[k] & 63);
      u[k] = at_node(up, up[k] & 63);
    }
#pragma unroll
    for (int k = 0; k < 2; k++)
      if (up[k] >= 0) {
        lo[k] |= l[k];
        hi[k] |= h[k];
        up[k] = u[k];
      }
  }
#pragma unroll
  for (int k = 0; k < 2; k++)
    bits[k] = static_cast<uint64_t>(static_cast<uint32_t>(hi[k])) << 32 |
              static_cast<uint32_t>(lo[k]);
}

// Whether one of the pages of slots first .. last-1 is out of range, as thread
// `at` of `step` sees it (first <= last, within the table).
__device__ __forceinline__ bool bad_pages(const Cache& c, int b, int first, int last, int at,
                                          int step) {
  if (first >= last) return false;
  const int end = (last - 1) / c.page_size;
  bool bad = false;
  for (int p = first / c.page_size + at; p <= end; p += step) {
    const int page = c.page_table[static_cast<int64_t>(b) * c.table_stride + p];
    bad |= page < 0 || page >= c.pages;
  }
  return bad;
}

// Host side ---------------------------------------------------------------

inline bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

inline bool strides_ok(int64_t a, int64_t b, int64_t c) {
  return a >= 0 && b >= 0 && c >= 0 && a % 8 == 0 && b % 8 == 0 && c % 8 == 0;
}

// The documented limits of a cache for B requests of N nodes.
inline specv_status check_cache(const specv_cache* c, int B, int N) {
  if (!c || !c->k || !c->v || !c->page_table || !c->lens) return SPECV_ERR_INVALID_ARG;
  if (c->dtype != SPECV_BF16 && c->dtype != SPECV_F16) return SPECV_ERR_INVALID_ARG;
  if (B < 1 || N < 1 || c->layers < 1 || c->pages < 1 || c->page_size < 1 || c->max_pages < 1 ||
      c->heads < 1 || c->head_dim < 1)
    return SPECV_ERR_INVALID_ARG;
  if (B > 1 && c->table_stride < c->max_pages) return SPECV_ERR_INVALID_ARG;
  if (B > SPECV_MAX_BATCH || N > SPECV_MAX_NODES || c->heads > 1024 ||
      c->head_dim > SPECV_MAX_HEAD_DIM || c->head_dim % 8 != 0)
    return SPECV_ERR_UNSUPPORTED;
  if (!aligned_to(c->k, 16) || !aligned_to(c->v, 16) || !aligned_to(c->page_table, 4) ||
      !aligned_to(c->lens, 4) || !strides_ok(c->layer_stride, 0, 0) ||
      !strides_ok(c->page_stride, c->row_stride, c->head_stride))
    return SPECV_ERR_INVALID_ARG;
  return SPECV_OK;
}

inline bool rows_ok(const specv_rows* r) {
  return r && r->data && aligned_to(r->data, 16) &&
         strides_ok(r->batch_stride, r->node_stride, r->head_stride);
}

inline Cache to_cache(const specv_cache* c) {
  return Cache{static_cast<uint16_t*>(c->k), static_cast<uint16_t*>(c->v), c->page_table, c->lens,
               c->layer_stride, c->page_stride, c->row_stride, c->head_stride, c->layers, c->pages,
               c->page_size, c->max_pages, c->table_stride, c->heads, c->head_dim};
}

inline Rows to_rows(const specv_rows* r) {
  return Rows{static_cast<uint16_t*>(r->data), r->batch_stride, r->node_stride, r->head_stride};
}

inline specv_status launched() {
  return cudaGetLastError() == cudaSuccess ? SPECV_OK : SPECV_ERR_CUDA;
}

}  // namespace specv_cache_ops
