// The paged cache's own operators: norms, rotation and append of a drafted
// tree's projections, and the move of the accepted path's rows.

#include "cache.cuh"

using namespace specv_cache_ops;

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;
constexpr double kInvTwoPi = 0.15915494309189533576888376337251;

// ------------------------------------------------------------------ append

constexpr int kAppendThreads = 256;
constexpr int kTokens = 4;                  // nodes a block takes
constexpr int kHalfMax = SPECV_MAX_HEAD_DIM / 2;

struct AppendParams {
  Cache cache;
  Rows q, k, v, q_out;
  const int32_t* parents;
  const int32_t* n_nodes;
  const uint16_t* q_weight;
  const uint16_t* k_weight;
  const float* inv_freq;
  int32_t* status;
  float eps, rope_scale;
  int N, q_heads, rot_dim, interleaved;
};

// A row of head_dim values is a group's: one lane to eight values, so that
// every load and store is 16 bytes.
template <class E, int kLanes>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams P) {
  constexpr int kGroups = kAppendThreads / kLanes;
  __shared__ int s_n, s_bad;
  __shared__ int s_pos[kMaxNodes];
  __shared__ float2 s_turn[kTokens][kHalfMax];
  __shared__ __align__(16) float s_x[kGroups][kLanes * 8];

  const int tid = threadIdx.x, lane = tid & 31;
  const int tiles = (P.N + kTokens - 1) / kTokens;
  const int b = blockIdx.x / tiles, first = (blockIdx.x % tiles) * kTokens;
  const Cache& C = P.cache;
  const int D = C.head_dim;

  if (tid < 32) {
    const int64_t slots = static_cast<int64_t>(C.max_pages) * C.page_size;
    Tree t = read_tree(P.parents, P.n_nodes, C.lens, b, P.N, slots, lane);
    if (!t.bad && __any_sync(kFullMask, bad_pages(C, b, t.len, t.len + t.n, lane, 32)))
      t.bad |= SPECV_DEV_BAD_CACHE;
    if (!t.bad) {
      int depth[2];
      depths(t, depth);
      s_pos[lane] = t.len + depth[0];
      s_pos[lane + 32] = t.len + depth[1];
    }
    if (lane == 0) {
      s_n = t.n;
      s_bad = t.bad;
      if (first == 0) P.status[b] = static_cast<int32_t>(t.bad);
    }
  }
  __syncthreads();
  const bool bad = s_bad != 0;
  const int n = s_n ? s_n : P.N;
  const int count = min(kTokens, n - first);
  if (count <= 0) return;

  // The angle of a far position loses its last digits in 32 bits (131072 radians
  // are known to 2^-7): the product and its remainder by 2 pi are taken in 64,
  // once for all heads; sincosf then sees at most pi.
  const int half = P.rot_dim / 2;
  if (!bad) {
    for (int e = tid; e < count * half; e += kAppendThreads) {
      const int t = e / half, j = e - t * half;
      const double a = static_cast<double>(s_pos[first + t]) * static_cast<double>(P.inv_freq[j]);
      const double r = fma(-rint(a * kInvTwoPi), kTwoPi, a);
      float sn, cs;
      sincosf(static_cast<float>(r), &sn, &cs);
      s_turn[t][j] = make_float2(cs * P.rope_scale, sn * P.rope_scale);
    }
  }
  __syncthreads();

  const int sub = tid % kLanes, group = tid / kLanes;
  const int d = sub * 8;
  const bool mine = d < D;
  float* x_row = s_x[group];
  const int heads = P.q_heads + 2 * C.heads;
  for (int r = group; r < count * heads; r += kGroups) {
    const int t = r / heads, h = r - t * heads, i = first + t;
    const bool is_q = h < P.q_heads, is_v = h >= P.q_heads + C.heads;
    const Rows& in = is_q ? P.q : is_v ? P.v : P.k;
    const int hh = is_q ? h : is_v ? h - P.q_heads - C.heads : h - P.q_heads;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (bad) {
      if (is_q && mine)
        *reinterpret_cast<uint4*>(P.q_out.data + b * P.q_out.batch_stride +
                                  i * P.q_out.node_stride + hh * P.q_out.head_stride + d) = w;
      continue;
    }
    if (mine)
      w = *reinterpret_cast<const uint4*>(in.data + b * in.batch_stride + i * in.node_stride +
                                          hh * in.head_stride + d);
    if (!is_v) {
      float x[8];
      const uint32_t* words = &w.x;
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const float2 f = E::unpack(words[e]);
        x[2 * e] = f.x;
        x[2 * e + 1] = f.y;
      }
      const uint16_t* weight = is_q ? P.q_weight : P.k_weight;
      const unsigned mask = kLanes == 32 ? kFullMask
                                         : ((1u << kLanes) - 1u) << (lane / kLanes * kLanes);
      if (weight) {
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; e++) sum = fmaf(x[e], x[e], sum);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o /= 2) sum += __shfl_xor_sync(mask, sum, o);
        const float inv = rsqrtf(sum / static_cast<float>(D) + P.eps);
        if (mine) {
          const uint4 g = *reinterpret_cast<const uint4*>(weight + d);
          const uint32_t* gw = &g.x;
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const float2 f = E::unpack(gw[e]);
            x[2 * e] = x[2 * e] * inv * f.x;
            x[2 * e + 1] = x[2 * e + 1] * inv * f.y;
          }
        }
      }
      if (P.interleaved) {
#pragma unroll
        for (int e = 0; e < 4; e++)
          if (d + 2 * e < P.rot_dim) {
            const float2 cs = s_turn[t][d / 2 + e];
            const float a = x[2 * e], c = x[2 * e + 1];
            x[2 * e] = a * cs.x - c * cs.y;
            x[2 * e + 1] = c * cs.x + a * cs.y;
          }
      } else if (half) {
        // the partner half a rotation away is another lane's
        __syncwarp(mask);
#pragma unroll
        for (int e = 0; e < 8; e++) x_row[d + e] = x[e];
        __syncwarp(mask);
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const int at = d + e;
          if (at < half) {
            const float2 cs = s_turn[t][at];
            x[e] = x[e] * cs.x - x_row[at + half] * cs.y;
          } else if (at < P.rot_dim) {
            const float2 cs = s_turn[t][at - half];
            x[e] = x[e] * cs.x + x_row[at - half] * cs.y;
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 4; e++) (&w.x)[e] = E::pack(x[2 * e], x[2 * e + 1]);
    }
    uint16_t* to;
    if (is_q)
      to = P.q_out.data + b * P.q_out.batch_stride + i * P.q_out.node_stride +
           hh * P.q_out.head_stride;
    else
      to = (is_v ? C.v : C.k) + C.slot(b, C.lens[b] + i) + hh * C.head_stride;
    if (mine) *reinterpret_cast<uint4*>(to + d) = w;
  }
}

// ------------------------------------------------------------------- keep

constexpr int kKeepThreads = 256;
constexpr int kBatch = 8;  // rows a thread has in flight

// One block per request and layer; a thread owns 16 bytes of a row of K or V
// and moves them for every kept node in order.  A path's nodes increase, so
// path[j] >= j: no row is a destination before it was read, also between the
// batches of loads (a destination j is below every later source).
__global__ void __launch_bounds__(kKeepThreads) keep_kernel(const Cache C, const int32_t* path_nodes,
                                                            const int32_t* accepted_len, int N,
                                                            int32_t* new_lens, int32_t* status) {
  __shared__ int64_t s_from[kMaxNodes], s_to[kMaxNodes];
  __shared__ int s_moves;
  const int tid = threadIdx.x, lane = tid & 31;
  const int b = blockIdx.x, layer = blockIdx.y;
  if (tid < 32) {
    int accepted = accepted_len[b];
    const int len = C.lens[b];
    unsigned bad = 0;
    if (accepted < 0 || accepted >= N) {
      bad |= SPECV_DEV_BAD_DRAFT_LEN;
      accepted = 0;
    }
    int last = 0;
    bool bad_path = false;
    int node[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 2; k++) {
      const int j = lane + 32 * k;
      if (j > accepted) continue;
      const int32_t* p = path_nodes + static_cast<int64_t>(b) * N + j;
      node[k] = p[0];
      bad_path |= j == 0 ? node[k] != 0 : node[k] <= p[-1] || node[k] >= N;
      last = max(last, node[k]);
    }
    last = __reduce_max_sync(kFullMask, last);
    if (__any_sync(kFullMask, bad_path)) bad |= SPECV_DEV_BAD_TREE;
    if (len < 0 || len > INT_MAX - 4 * kMaxNodes ||
        (!bad && static_cast<int64_t>(len) + last >= static_cast<int64_t>(C.max_pages) * C.page_size))
      bad |= SPECV_DEV_BAD_CACHE;
    bool bad_page = false;
    if (!bad) {
      // the pages of the rows that move, and no others
#pragma unroll
      for (int k = 0; k < 2; k++) {
        const int j = lane + 32 * k;
        if (j < 1 || j > accepted) continue;
        bad_page |= bad_pages(C, b, len + node[k], len + node[k] + 1, 0, 1) ||
                    bad_pages(C, b, len + j, len + j + 1, 0, 1);
      }
    }
    if (__any_sync(kFullMask, bad_page)) bad |= SPECV_DEV_BAD_CACHE;
    if (!bad) {
#pragma unroll
      for (int k = 0; k < 2; k++) {
        const int j = lane + 32 * k;
        if (j < 1 || j > accepted) continue;
        s_from[j - 1] = C.slot(b, len + node[k]);
        s_to[j - 1] = C.slot(b, len + j);
      }
    }
    if (lane == 0) {
      s_moves = bad ? 0 : accepted;
      if (layer == 0) {
        status[b] = static_cast<int32_t>(bad);
        new_lens[b] = bad ? len : len + accepted + 1;
      }
    }
  }
  __syncthreads();
  const int moves = s_moves;
  if (moves == 0) return;
  const int per_row = C.heads * (C.head_dim / 8);
  for (int u = tid; u < 2 * per_row; u += kKeepThreads) {
    const int at = u < per_row ? u : u - per_row;
    const int h = at / (C.head_dim / 8), d = (at - h * (C.head_dim / 8)) * 8;
    uint16_t* base = (u < per_row ? C.k : C.v) + layer * C.layer_stride + h * C.head_stride + d;
    for (int j0 = 0; j0 < moves; j0 += kBatch) {
      uint4 w[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; j++)
        if (j0 + j < moves) w[j] = *reinterpret_cast<const uint4*>(base + s_from[j0 + j]);
#pragma unroll
      for (int j = 0; j < kBatch; j++)
        if (j0 + j < moves) *reinterpret_cast<uint4*>(base + s_to[j0 + j]) = w[j];
    }
  }
}

}  // namespace

extern "C" {

specv_status spec_append_nodes(const specv_cache* cache, const specv_rows* q, const specv_rows* k,
                               const specv_rows* v, const int32_t* parents,
                               const int32_t* n_nodes, int B, int N, int q_heads,
                               const void* q_weight, const void* k_weight, float eps,
                               const float* inv_freq, int rot_dim, int interleaved,
                               float rope_scale, const specv_rows* q_out, int32_t* status,
                               specv_stream_t stream) {
  const specv_status s = check_cache(cache, B, N);
  if (s != SPECV_OK) return s;
  if (!rows_ok(q) || !rows_ok(k) || !rows_ok(v) || !rows_ok(q_out) || !status || q_heads < 1 ||
      rot_dim < 0 || rot_dim % 2 != 0 || rot_dim > cache->head_dim || (rot_dim > 0) != !!inv_freq ||
      cache->layers != 1)
    return SPECV_ERR_INVALID_ARG;
  if (!aligned_to(parents, 4) || !aligned_to(n_nodes, 4) || !aligned_to(q_weight, 16) ||
      !aligned_to(k_weight, 16) || !aligned_to(inv_freq, 4) || !aligned_to(status, 4))
    return SPECV_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || eps > 3e38f || !(rope_scale > -3e38f && rope_scale < 3e38f))
    return SPECV_ERR_INVALID_ARG;
  if (q_heads > 1024) return SPECV_ERR_UNSUPPORTED;
  const AppendParams P{to_cache(cache),
                       to_rows(q),
                       to_rows(k),
                       to_rows(v),
                       to_rows(q_out),
                       parents,
                       n_nodes,
                       static_cast<const uint16_t*>(q_weight),
                       static_cast<const uint16_t*>(k_weight),
                       inv_freq,
                       status,
                       eps,
                       rope_scale,
                       N,
                       q_heads,
                       rot_dim,
                       interleaved};
  const unsigned grid = static_cast<unsigned>(B) * ((N + kTokens - 1) / kTokens);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool narrow = cache->head_dim <= 64;
  if (cache->dtype == SPECV_BF16) {
    if (narrow) append_kernel<Bf16, 8><<<grid, kAppendThreads, 0, st>>>(P);
    else append_kernel<Bf16, 16><<<grid, kAppendThreads, 0, st>>>(P);
  } else {
    if (narrow) append_kernel<F16, 8><<<grid, kAppendThreads, 0, st>>>(P);
    else append_kernel<F16, 16><<<grid, kAppendThreads, 0, st>>>(P);
  }
  return launched();
}

specv_status spec_keep_path(const specv_cache* cache, const int32_t* path_nodes,
                            const int32_t* accepted_len, int B, int N, int32_t* new_lens,
                            int32_t* status, specv_stream_t stream) {
  const specv_status s = check_cache(cache, B, N);
  if (s != SPECV_OK) return s;
  if (!path_nodes || !accepted_len || !new_lens || !status || new_lens == cache->lens ||
      !aligned_to(path_nodes, 4) || !aligned_to(accepted_len, 4) || !aligned_to(new_lens, 4) ||
      !aligned_to(status, 4))
    return SPECV_ERR_INVALID_ARG;
  if (cache->layers > 65535) return SPECV_ERR_UNSUPPORTED;
  keep_kernel<<<dim3(static_cast<unsigned>(B), static_cast<unsigned>(cache->layers)), kKeepThreads,
                0, reinterpret_cast<cudaStream_t>(stream)>>>(to_cache(cache), path_nodes,
                                                             accepted_len, N, new_lens, status);
  return launched();
}

}  // extern "C"
