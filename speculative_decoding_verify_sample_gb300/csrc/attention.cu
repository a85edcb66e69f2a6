// Attention of a drafted tree's nodes over the paged cache.

#include "cache.cuh"

using namespace specv_cache_ops;

namespace {

// ----------------------------------------------------------------- prepare

constexpr int kPrepThreads = 128;

// What the attention kernel reads of a request: its keys (0 where the request
// is flagged), its nodes and each node's ancestors.
struct Plan {
  int32_t* len;       // [B] verified tokens
  int32_t* nodes;     // [B] rows to write; flagged: ~rows (all become 0)
  uint64_t* visible;  // [B][kMaxNodes] bit j: node sees node j
};

__global__ void __launch_bounds__(kPrepThreads) prepare_kernel(const Cache C, const int32_t* parents,
                                                               const int32_t* n_nodes, int N,
                                                               Plan plan, int32_t* status) {
  __shared__ int s_n, s_len, s_bad;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  Tree t;
  if (tid < 32) {
    t = read_tree(parents, n_nodes, C.lens, b, N, static_cast<int64_t>(C.max_pages) * C.page_size,
                  lane);
    if (lane == 0) {
      s_n = t.n;
      s_len = t.len;
      s_bad = t.bad;
    }
  }
  __syncthreads();
  const bool bad_page =
      !s_bad && bad_pages(C, b, 0, s_len + s_n, tid, kPrepThreads);
  const bool any = __syncthreads_or(bad_page);
  if (tid < 32) {
    if (any) t.bad |= SPECV_DEV_BAD_CACHE;
    if (!t.bad) {
      uint64_t bits[2];
      ancestors(t, lane, bits);
      plan.visible[b * kMaxNodes + lane] = bits[0];
      plan.visible[b * kMaxNodes + lane + 32] = bits[1];
    }
    if (lane == 0) {
      plan.len[b] = t.bad ? 0 : t.len;
      plan.nodes[b] = t.bad ? ~(t.n ? t.n : N) : t.n;
      status[b] = static_cast<int32_t>(t.bad);
    }
  }
}

// --------------------------------------------------------------- attention

struct AttnParams {
  Cache cache;
  Rows q, out;
  Plan plan;
  int N, q_heads;
  float scale_log2;
};

// One warp per output row, online softmax over the slots in order; lane l has
// the values d = 4 l .. 4 l + 3 of the head.
template <class E>
__global__ void __launch_bounds__(128) attention_kernel(const AttnParams P, int rows) {
  const int row = (blockIdx.x * 128 + threadIdx.x) / 32, lane = threadIdx.x & 31;
  if (row >= rows) return;
  const Cache& C = P.cache;
  const int h = row % P.q_heads, i = row / P.q_heads % P.N, b = row / P.q_heads / P.N;
  int n = P.plan.nodes[b];
  const bool bad = n < 0;
  if (bad) n = ~n;
  if (i >= n) return;
  const int d = 4 * lane;
  const bool mine = d < C.head_dim;
  uint2* to = reinterpret_cast<uint2*>(P.out.data + b * P.out.batch_stride + i * P.out.node_stride +
                                       h * P.out.head_stride + d);
  if (bad) {
    if (mine) *to = make_uint2(0, 0);
    return;
  }
  const int kvh = h / (P.q_heads / C.heads);
  float q[4] = {0, 0, 0, 0}, o[4] = {0, 0, 0, 0};
  if (mine) {
    const uint2 w = *reinterpret_cast<const uint2*>(
        P.q.data + b * P.q.batch_stride + i * P.q.node_stride + h * P.q.head_stride + d);
    const float2 f = E::unpack(w.x), g = E::unpack(w.y);
    q[0] = f.x, q[1] = f.y, q[2] = g.x, q[3] = g.y;
  }
  const int len = P.plan.len[b];
  const uint64_t visible = P.plan.visible[b * kMaxNodes + i];
  float m = -INFINITY, l = 0.0f;
  for (int s = 0; s < len + n; s++) {
    if (s >= len && !(visible >> (s - len) & 1)) continue;
    const int64_t at = C.slot(b, s) + kvh * C.head_stride + d;
    float k[4] = {0, 0, 0, 0}, v[4] = {0, 0, 0, 0};
    if (mine) {
      const uint2 kw = *reinterpret_cast<const uint2*>(C.k + at);
      const uint2 vw = *reinterpret_cast<const uint2*>(C.v + at);
      float2 f = E::unpack(kw.x), g = E::unpack(kw.y);
      k[0] = f.x, k[1] = f.y, k[2] = g.x, k[3] = g.y;
      f = E::unpack(vw.x), g = E::unpack(vw.y);
      v[0] = f.x, v[1] = f.y, v[2] = g.x, v[3] = g.y;
    }
    float x = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
    for (int off = 16; off > 0; off /= 2) x += __shfl_xor_sync(kFullMask, x, off);
    x *= P.scale_log2;
    const float top = fmaxf(m, x);
    const float base = top == -INFINITY ? 0.0f : top;
    const float old = exp2f(m - base), p = exp2f(x - base);
    l = l * old + p;
#pragma unroll
    for (int e = 0; e < 4; e++) o[e] = o[e] * old + p * v[e];
    m = top;
  }
  const float inv = 1.0f / l;
  if (mine) *to = make_uint2(E::pack(o[0] * inv, o[1] * inv), E::pack(o[2] * inv, o[3] * inv));
}

// ------------------------------------------------------------------- host

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

struct Layout {
  size_t len, nodes, visible, total;
};

Layout layout(int B) {
  Layout w;
  w.len = 0;
  w.nodes = align256(static_cast<size_t>(B) * 4);
  w.visible = w.nodes + align256(static_cast<size_t>(B) * 4);
  w.total = w.visible + align256(static_cast<size_t>(B) * kMaxNodes * 8);
  return w;
}

}  // namespace

extern "C" {

size_t specv_attention_workspace_bytes(int B, int N, int q_heads, int kv_heads, int head_dim) {
  if (B < 1 || B > SPECV_MAX_BATCH || N < 1 || N > SPECV_MAX_NODES || kv_heads < 1 ||
      q_heads < kv_heads || q_heads > 1024 || q_heads % kv_heads != 0 || head_dim < 8 ||
      head_dim > SPECV_MAX_HEAD_DIM || head_dim % 8 != 0)
    return 0;
  return layout(B).total;
}

specv_status spec_tree_attention(const specv_cache* cache, const specv_rows* q,
                                 const int32_t* parents, const int32_t* n_nodes, int B, int N,
                                 int q_heads, float scale, const specv_rows* out, int32_t* status,
                                 void* workspace, size_t workspace_bytes, specv_stream_t stream) {
  const specv_status s = check_cache(cache, B, N);
  if (s != SPECV_OK) return s;
  if (!rows_ok(q) || !rows_ok(out) || !status || !workspace || cache->layers != 1 || q_heads < 1 ||
      q_heads % cache->heads != 0 || !(scale > 0.0f) || scale > 3e38f)
    return SPECV_ERR_INVALID_ARG;
  if (!aligned_to(parents, 4) || !aligned_to(n_nodes, 4) || !aligned_to(status, 4) ||
      !aligned_to(workspace, 256))
    return SPECV_ERR_INVALID_ARG;
  if (q_heads > 1024) return SPECV_ERR_UNSUPPORTED;
  const Layout w = layout(B);
  if (workspace_bytes < w.total) return SPECV_ERR_WORKSPACE;
  char* base = static_cast<char*>(workspace);
  const Plan plan{reinterpret_cast<int32_t*>(base + w.len),
                  reinterpret_cast<int32_t*>(base + w.nodes),
                  reinterpret_cast<uint64_t*>(base + w.visible)};
  const Cache C = to_cache(cache);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  prepare_kernel<<<B, kPrepThreads, 0, st>>>(C, parents, n_nodes, N, plan, status);
  const AttnParams P{C, to_rows(q), to_rows(out), plan, N, q_heads, scale * 1.4426950408889634f};
  const int rows = B * N * q_heads;
  const unsigned grid = (static_cast<unsigned>(rows) + 3) / 4;
  if (cache->dtype == SPECV_BF16) attention_kernel<Bf16><<<grid, 128, 0, st>>>(P, rows);
  else attention_kernel<F16><<<grid, 128, 0, st>>>(P, rows);
  return launched();
}

}  // extern "C"
