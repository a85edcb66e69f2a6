// The paged cache's own operators: norms, rotation and append of a drafted
// tree's or a chunk's projections, and the move of the accepted path's rows.

#include "cache.cuh"

using namespace specv_cache_ops;

namespace {

// ------------------------------------------------------------------ append

constexpr int kAppendWarps = 8;
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
  int B, N, q_heads, rot_dim, interleaved;
};

// cos and sin of pos * freq.  The angle of a far position loses its last digits
// in 32 bits (near 131072 radians they are 2^-7 apart), so it is taken in turns:
// the frequency's fraction of a turn as a 64-bit whole number, whose product
// with the position drops whole turns by itself and keeps the top 32 bits.
__device__ __forceinline__ uint64_t steps_of(float freq) {
  const double turns = static_cast<double>(freq) * 0.15915494309189533576888;
  const double part = turns - floor(turns);  // [0, 1): 1 itself, by rounding, is no turn
  return part < 1.0 ? static_cast<uint64_t>(part * 18446744073709551616.0) : 0;
}

__device__ __forceinline__ float2 turn(int pos, float freq, uint64_t steps, float scale) {
  const int top = static_cast<int>(static_cast<uint32_t>(steps * static_cast<uint64_t>(pos) >> 32));
  float sn, cs;
  sincospif(static_cast<float>(top) * 4.656612873077393e-10f, &sn, &cs);  // 2^-31 half turns
  if (!isfinite(freq)) sn = cs = NAN;
  return make_float2(cs * scale, sn * scale);
}

// x <- x / sqrt(mean x^2 + eps) * weight, then the pairs' rotation, in 32 bits.
// Each row is read and written once: 256 trees of 17 to 32 nodes, 64 query and 8 + 8
// key and value heads of 128, 57 us (257 MB, 4.5 TB/s).  Three blocks of 80 registers fit an
// SM, 456 the machine, and a wave that is not full costs nearly a whole one (of 32 nodes:
// 114 trees, one wave, 31.5 us, 128 43.2; 228 56.5, 256 65.9); under the profiler 71 % of the
// issue slots are taken.  32 trees 10 to 12 us and one chain 6 to 8, most of it
// the chain of loads from a request's length to its slot.
//
// A warp has a node and goes through its heads, 32 / kLanes rows at a time.  A
// lane has two 16-byte pieces of a row, the two that a rotation in halves
// joins, and their cosines and sines stay in its registers for all heads.
// kOdd: the halves do not begin at a piece; their elements meet in shared memory.
template <class E, int kLanes, bool kOdd>
__global__ void __launch_bounds__(kAppendWarps * 32, 3) append_kernel(const AppendParams P) {
  constexpr int kRowsAtOnce = 32 / kLanes;
  constexpr int kStages = kOdd ? 2 : 4;  // passes of a warp in shared memory
  __shared__ float2 s_turn[kAppendWarps][kHalfMax];
  __shared__ uint4 s_in[kAppendWarps][kStages][2][32];
  __shared__ __align__(16) float s_x[kOdd ? kAppendWarps * kRowsAtOnce : 1][kOdd ? kLanes * 16 : 4];

  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int token = blockIdx.x * kAppendWarps + warp;
  const int b = token / P.N, i = token - b * P.N;
  if (b >= P.B) return;
  const Cache& C = P.cache;
  const int pieces = C.head_dim / 8, half = P.rot_dim / 2;
  const int sub = lane % kLanes, group = lane / kLanes;
  // this lane's pieces of a row; behind the last: none
  int piece[2];
  if (!kOdd && !P.interleaved && sub < half / 8) {
    piece[0] = sub;
    piece[1] = sub + half / 8;
  } else {
    const int done = kOdd || P.interleaved ? 0 : half / 8, left = pieces - 2 * done;
    piece[0] = sub - done < (left + 1) / 2 ? done + sub : pieces;
    piece[1] = sub - done < left / 2 ? piece[0] + (left + 1) / 2 : pieces;
  }
  const bool mine[2] = {piece[0] < pieces, piece[1] < pieces};

  // Passes over the heads: queries, keys, values, each kRowsAtOnce rows.
  const int q_passes = (P.q_heads + kRowsAtOnce - 1) / kRowsAtOnce;
  const int kv_passes = (C.heads + kRowsAtOnce - 1) / kRowsAtOnce;
  const int passes = q_passes + 2 * kv_passes;
  // A lane copies and reads its own places, so nothing but its own wait orders them.
  auto load = [&](int p, int stage) {
    const bool is_q = p < q_passes, is_k = p < q_passes + kv_passes;
    const Rows& in = is_q ? P.q : is_k ? P.k : P.v;
    const int h = (is_q ? p : is_k ? p - q_passes : p - q_passes - kv_passes) * kRowsAtOnce + group;
    const bool real = p < passes && h < (is_q ? P.q_heads : C.heads);
    const uint16_t* from = in.data + b * in.batch_stride + i * in.node_stride + h * in.head_stride;
#pragma unroll
    for (int k = 0; k < 2; k++) {
      const bool some = real && mine[k];
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(static_cast<uint32_t>(
                       __cvta_generic_to_shared(&s_in[warp][stage][k][lane]))),
                   "l"(some ? from + piece[k] * 8 : in.data), "r"(some ? 16 : 0)
                   : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int p = blockIdx.y;
#pragma unroll
  for (int k = 0; k < kStages - 1; k++) load(p + k * gridDim.y, k);  // while the request is checked

  float freq[2];
  uint64_t steps[2];
#pragma unroll
  for (int k = 0; k < 2; k++) {
    freq[k] = lane + 32 * k < half ? P.inv_freq[lane + 32 * k] : 0.0f;
    steps[k] = steps_of(freq[k]);
  }
  Tree t = read_tree(P.parents, P.n_nodes, C.lens, b, P.N,
                     static_cast<int64_t>(C.max_pages) * C.page_size, lane);
  if (!t.bad && __any_sync(kFullMask, bad_pages(C, b, t.len, t.len + t.n, lane, 32)))
    t.bad |= SPECV_DEV_BAD_CACHE;
  if (i == 0 && blockIdx.y == 0 && lane == 0) P.status[b] = static_cast<int32_t>(t.bad);
  if (t.bad || i >= t.n) asm volatile("cp.async.wait_all;" ::: "memory");
  if (i >= (t.n ? t.n : P.N)) return;
  if (t.bad) {  // a flagged request: queries become 0, the cache stays
    for (; p < q_passes; p += gridDim.y)
#pragma unroll
      for (int k = 0; k < 2; k++) {
        const int h = p * kRowsAtOnce + group;
        if (mine[k] && h < P.q_heads)
          *reinterpret_cast<uint4*>(P.q_out.data + b * P.q_out.batch_stride +
                                    i * P.q_out.node_stride + h * P.q_out.head_stride +
                                    piece[k] * 8) = make_uint4(0, 0, 0, 0);
      }
    return;
  }

  const int64_t slot = C.slot(b, t.len + i);
  float2 cs[2][4];  // of this lane's pairs: four of each piece, or eight of both
  if (half) {
    int depth[2];
    depths(t, depth);
    const int pos = t.len + at_node(depth, i);
#pragma unroll
    for (int k = 0; k < 2; k++)
      if (lane + 32 * k < half)
        s_turn[warp][lane + 32 * k] = turn(pos, freq[k], steps[k], P.rope_scale);
    __syncwarp();
    if (!kOdd) {
#pragma unroll
      for (int k = 0; k < 2; k++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const int j = P.interleaved ? piece[k] * 4 + e : piece[0] * 8 + 4 * k + e;
          cs[k][e] = mine[k] && j < half ? s_turn[warp][j] : make_float2(1.0f, 0.0f);
        }
    }
  }
  const bool joined = !kOdd && !P.interleaved && sub < half / 8;

  int kind = -1;  // 0 queries, 1 keys, 2 values
  const uint16_t* weight = nullptr;
  uint4 g[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  for (int stage = 0; p < passes; p += gridDim.y, stage = (stage + 1) % kStages) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    uint4 w[2] = {s_in[warp][stage][0][lane], s_in[warp][stage][1][lane]};
    load(p + (kStages - 1) * gridDim.y, (stage + kStages - 1) % kStages);  // read a pass ago
    const int now = p < q_passes ? 0 : p < q_passes + kv_passes ? 1 : 2;
    const int h = (now == 0 ? p : now == 1 ? p - q_passes : p - q_passes - kv_passes) * kRowsAtOnce + group;
    if (now != kind) {
      kind = now;
      weight = kind == 0 ? P.q_weight : kind == 1 ? P.k_weight : nullptr;
      if (weight)
#pragma unroll
        for (int k = 0; k < 2; k++)
          if (mine[k]) g[k] = *reinterpret_cast<const uint4*>(weight + piece[k] * 8);
    }
    if (kind < 2 && (weight || half)) {
      float x[2][8];
#pragma unroll
      for (int k = 0; k < 2; k++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const float2 f = E::unpack((&w[k].x)[e]);
          x[k][2 * e] = f.x;
          x[k][2 * e + 1] = f.y;
        }
      if (weight) {
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 2; k++)
#pragma unroll
          for (int e = 0; e < 8; e++) sum = fmaf(x[k][e], x[k][e], sum);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o /= 2) sum += __shfl_xor_sync(kFullMask, sum, o);
        const float inv = rsqrtf(sum / static_cast<float>(C.head_dim) + P.eps);
#pragma unroll
        for (int k = 0; k < 2; k++)
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const float2 f = E::unpack((&g[k].x)[e]);
            x[k][2 * e] = x[k][2 * e] * inv * f.x;
            x[k][2 * e + 1] = x[k][2 * e + 1] * inv * f.y;
          }
      }
      if (kOdd) {
        float* row = s_x[warp * kRowsAtOnce + group];
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 2; k++)
          if (mine[k]) {
            *reinterpret_cast<float4*>(row + piece[k] * 8) =
                make_float4(x[k][0], x[k][1], x[k][2], x[k][3]);
            *reinterpret_cast<float4*>(row + piece[k] * 8 + 4) =
                make_float4(x[k][4], x[k][5], x[k][6], x[k][7]);
          }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 2; k++)
#pragma unroll
          for (int e = 0; e < 8; e++) {
            const int d = piece[k] * 8 + e;
            if (!mine[k] || d >= P.rot_dim) continue;
            const float2 c = s_turn[warp][d < half ? d : d - half];
            x[k][e] = d < half ? x[k][e] * c.x - row[d + half] * c.y
                               : x[k][e] * c.x + row[d - half] * c.y;
          }
      } else if (P.interleaved) {
        if (half)
#pragma unroll
          for (int k = 0; k < 2; k++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const float a = x[k][2 * e], c = x[k][2 * e + 1];
              if (piece[k] * 4 + e < half) {
                x[k][2 * e] = a * cs[k][e].x - c * cs[k][e].y;
                x[k][2 * e + 1] = c * cs[k][e].x + a * cs[k][e].y;
              }
            }
      } else if (joined) {
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const float2 f = cs[e / 4][e % 4];
          const float a = x[0][e], c = x[1][e];
          x[0][e] = a * f.x - c * f.y;
          x[1][e] = c * f.x + a * f.y;
        }
      }
#pragma unroll
      for (int k = 0; k < 2; k++)
#pragma unroll
        for (int e = 0; e < 4; e++) (&w[k].x)[e] = E::pack(x[k][2 * e], x[k][2 * e + 1]);
    }
    uint16_t* to = kind == 0 ? P.q_out.data + b * P.q_out.batch_stride + i * P.q_out.node_stride +
                                   h * P.q_out.head_stride
                             : (kind == 1 ? C.k : C.v) + slot + h * C.head_stride;
#pragma unroll
    for (int k = 0; k < 2; k++)
      if (mine[k] && h < (kind == 0 ? P.q_heads : C.heads))
        *reinterpret_cast<uint4*>(to + piece[k] * 8) = w[k];
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <class E>
void run_append(const AppendParams& P, cudaStream_t stream) {
  const int half = P.rot_dim / 2;
  const bool odd = half % 8 != 0 && !P.interleaved, narrow = P.cache.head_dim <= 64;
  const int rows_at_once = narrow ? 8 : 4;
  const int passes = (P.q_heads + rows_at_once - 1) / rows_at_once +
                     2 * ((P.cache.heads + rows_at_once - 1) / rows_at_once);
  // Few nodes: their heads are shared out over several warps, 16 to an SM (48 trees,
  // 1,536 nodes, 12.4 us with two warps a node and 14.4 with one; 64 trees, 2,048 nodes,
  // 15.0 and 16.0; for 32 to an SM 32 trees took 13.8 us against 11.6, 64 trees 18.2).
  const int tokens = P.B * P.N;
  const int splits = tokens >= 16 * kSms ? 1 : (16 * kSms + tokens - 1) / tokens;
  const dim3 grid((tokens + kAppendWarps - 1) / kAppendWarps, splits < passes ? splits : passes);
  constexpr int kThreads = kAppendWarps * 32;
  if (narrow) {
    if (odd) append_kernel<E, 4, true><<<grid, kThreads, 0, stream>>>(P);
    else append_kernel<E, 4, false><<<grid, kThreads, 0, stream>>>(P);
  } else {
    if (odd) append_kernel<E, 8, true><<<grid, kThreads, 0, stream>>>(P);
    else append_kernel<E, 8, false><<<grid, kThreads, 0, stream>>>(P);
  }
}

// ---------------------------------------------------------- append a chunk

struct ChunkParams {
  AppendParams a;  // of it not parents, n_nodes, N; rows are packed
  const int32_t* cu_tokens;
  const int32_t* positions;  // [axes, T], NULL: the slot is the position
  const int32_t* axis_of;    // [rot_dim / 2]
  int64_t position_stride;
  int T, axes;
  int each, slices;  // tokens of a warp, warps that share a token's heads
};

// One request of a packed batch, as a warp holds it.
struct Packed {
  int first, last, len;  // its rows first .. last-1 (none: last = first)
  unsigned bad;
};

// Reads and checks request b (every lane of a warp calls this).
__device__ __forceinline__ Packed read_packed(const ChunkParams& P, int b, unsigned bad, int lane) {
  const Cache& C = P.a.cache;
  Packed r;
  r.first = P.cu_tokens[b];
  r.last = P.cu_tokens[b + 1];
  r.len = C.lens[b];
  r.bad = bad;
  if (r.first < 0 || r.last < r.first || r.last > P.T) {
    r.bad |= SPECV_DEV_BAD_DRAFT_LEN;
    r.last = r.first;
  }
  const int64_t end = static_cast<int64_t>(r.len) + (r.last - r.first);
  if (r.len < 0 || end > INT_MAX - 1024 || end > static_cast<int64_t>(C.max_pages) * C.page_size)
    r.bad |= SPECV_DEV_BAD_CACHE;
  if (!r.bad &&
      __any_sync(kFullMask, bad_pages(C, b, r.len, static_cast<int>(end), lane, 32)))
    r.bad |= SPECV_DEV_BAD_CACHE;
  return r;
}

// The request that has packed row t, -1: none.  The last one that begins at or before t
// (32 places at a time, so three steps for 32,768 requests); where cu_tokens falls that
// may be another, and all are looked at.
__device__ __forceinline__ int request_of(const ChunkParams& P, int t, int lane) {
  int lo = 0, hi = P.a.B;  // cu_tokens[lo] <= t if any is, cu_tokens[hi] > t if any is
  while (hi - lo > 1) {
    const int step = (hi - lo + 32) / 33;
    const int at = lo + (lane + 1) * step;
    const unsigned before = __ballot_sync(kFullMask, at < hi && P.cu_tokens[at] <= t);
    const int n = __popc(before);
    hi = min(hi, lo + (n + 1) * step);
    lo += n * step;
  }
  auto has = [&](int b) { return P.cu_tokens[b] <= t && t < P.cu_tokens[b + 1]; };
  if (has(lo)) return lo;
  for (int b0 = 0; b0 < P.a.B; b0 += 32) {
    const unsigned found = __ballot_sync(kFullMask, b0 + lane < P.a.B && has(b0 + lane));
    if (found) return b0 + __ffs(found) - 1;
  }
  return -1;
}

// The same norm and rotation for packed tokens of any number, whose pairs may turn by
// the positions of several axes.
//
// Each row is read and written once: 16 requests of 513 to 4,093 tokens, three axes, 168 us
// (906 MB, 5.4 TB/s, 0.80 of a plain copy); one of 517 tokens 10.3 us, launch and the chain to a
// token's slot and angles; a single token of each of 64, 256 and 1,024 requests 8.3, 10.4, 14.4.
// With 24, 48, 72 and 144 warps to an SM in the grid the first took
// 168, 181, 166 and 168.
//
// A warp has `each` tokens in a row (or every slices-th pass of them), and its copies
// run kStages - 1 passes ahead through all of them: they need no more than the
// token's number, so the chain from a token to its request, slot and angles passes while
// they are under way.  Lanes and pieces as in append_kernel.
template <class E, int kLanes, bool kOdd>
__global__ void __launch_bounds__(kAppendWarps * 32, 3) append_chunk_kernel(const ChunkParams P) {
  constexpr int kRowsAtOnce = 32 / kLanes;
  constexpr int kStages = kOdd ? 2 : 4;  // passes of a warp in shared memory
  __shared__ float2 s_turn[kAppendWarps][kHalfMax];
  __shared__ uint4 s_in[kAppendWarps][kStages][2][32];
  __shared__ __align__(16) float s_x[kOdd ? kAppendWarps * kRowsAtOnce : 1][kOdd ? kLanes * 16 : 4];

  const AppendParams& A = P.a;
  const Cache& C = A.cache;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int global = blockIdx.x * kAppendWarps + warp, warps = gridDim.x * kAppendWarps;
  const int pieces = C.head_dim / 8, half = A.rot_dim / 2;
  const int sub = lane % kLanes, group = lane / kLanes;
  // this lane's pieces of a row; behind the last: none
  int piece[2];
  if (!kOdd && !A.interleaved && sub < half / 8) {
    piece[0] = sub;
    piece[1] = sub + half / 8;
  } else {
    const int done = kOdd || A.interleaved ? 0 : half / 8, left = pieces - 2 * done;
    piece[0] = sub - done < (left + 1) / 2 ? done + sub : pieces;
    piece[1] = sub - done < left / 2 ? piece[0] + (left + 1) / 2 : pieces;
  }
  const bool mine[2] = {piece[0] < pieces, piece[1] < pieces};
  const bool joined = !kOdd && !A.interleaved && sub < half / 8;

  // Passes over a token's heads: queries, keys, values, each kRowsAtOnce rows.
  const int q_passes = (A.q_heads + kRowsAtOnce - 1) / kRowsAtOnce;
  const int kv_passes = (C.heads + kRowsAtOnce - 1) / kRowsAtOnce;
  const int passes = q_passes + 2 * kv_passes;
  const int slice = global % P.slices;
  const int64_t begin = static_cast<int64_t>(global / P.slices) * P.each;
  const int t0 = static_cast<int>(min(begin, static_cast<int64_t>(P.T)));
  const int t1 = static_cast<int>(min(begin + P.each, static_cast<int64_t>(P.T)));
  // A lane copies and reads its own places, so nothing but its own wait orders them.
  int ahead_t = t0, ahead_p = slice;
  auto load = [&](int stage) {
    const int p = ahead_p;
    const bool is_q = p < q_passes, is_k = p < q_passes + kv_passes;
    const Rows& in = is_q ? A.q : is_k ? A.k : A.v;
    const int h = (is_q ? p : is_k ? p - q_passes : p - q_passes - kv_passes) * kRowsAtOnce + group;
    const bool real = ahead_t < t1 && p < passes && h < (is_q ? A.q_heads : C.heads);
    const uint16_t* from = in.data + ahead_t * in.node_stride + h * in.head_stride;
#pragma unroll
    for (int k = 0; k < 2; k++) {
      const bool some = real && mine[k];
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(static_cast<uint32_t>(
                       __cvta_generic_to_shared(&s_in[warp][stage][k][lane]))),
                   "l"(some ? from + piece[k] * 8 : in.data), "r"(some ? 16 : 0)
                   : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ahead_p += P.slices;
    if (ahead_p >= passes) {
      ahead_p = slice;
      ahead_t++;
    }
  };
#pragma unroll
  for (int k = 0; k < kStages - 1; k++) load(k);

  float freq[2];
  uint64_t steps[2];
  int axis[2] = {0, 0};
  bool off_axis = false;
#pragma unroll
  for (int k = 0; k < 2; k++) {
    const int j = lane + 32 * k;
    freq[k] = j < half ? A.inv_freq[j] : 0.0f;
    steps[k] = steps_of(freq[k]);
    if (P.axis_of && j < half) {
      axis[k] = P.axis_of[j];
      off_axis |= axis[k] < 0 || axis[k] >= P.axes;
    }
  }
  const unsigned call_bad = __any_sync(kFullMask, off_axis) ? SPECV_DEV_BAD_POSITION : 0;

  int b = -1, stage = 0;
  Packed r{0, 0, 0, 0};
  for (int t = t0; t < t1; t++) {
    if (b < 0 || t >= r.last) {
      b = request_of(P, t, lane);
      if (b >= 0) r = read_packed(P, b, call_bad, lane);
    }
    const bool writes = b >= 0 && !r.bad;
    const int at = r.len + t - r.first;
    const int64_t slot = writes ? C.slot(b, at) : 0;
    float2 cs[2][4];  // of this lane's pairs: four of each piece, or eight of both
    if (half && writes) {
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 2; k++)
        if (lane + 32 * k < half) {
          const int pos = P.positions ? P.positions[axis[k] * P.position_stride + t] : at;
          s_turn[warp][lane + 32 * k] = turn(pos, freq[k], steps[k], A.rope_scale);
        }
      __syncwarp();
      if (!kOdd) {
#pragma unroll
        for (int k = 0; k < 2; k++)
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const int j = A.interleaved ? piece[k] * 4 + e : piece[0] * 8 + 4 * k + e;
            cs[k][e] = mine[k] && j < half ? s_turn[warp][j] : make_float2(1.0f, 0.0f);
          }
      }
    }

    int kind = -1;  // 0 queries, 1 keys, 2 values
    const uint16_t* weight = nullptr;
    uint4 g[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    for (int p = slice; p < passes; p += P.slices, stage = (stage + 1) % kStages) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      uint4 w[2] = {s_in[warp][stage][0][lane], s_in[warp][stage][1][lane]};
      load((stage + kStages - 1) % kStages);  // read a pass ago
      const int now = p < q_passes ? 0 : p < q_passes + kv_passes ? 1 : 2;
      const int h = (now == 0 ? p : now == 1 ? p - q_passes : p - q_passes - kv_passes) * kRowsAtOnce + group;
      if (now != kind) {
        kind = now;
        weight = kind == 0 ? A.q_weight : kind == 1 ? A.k_weight : nullptr;
        if (weight)
#pragma unroll
          for (int k = 0; k < 2; k++)
            if (mine[k]) g[k] = *reinterpret_cast<const uint4*>(weight + piece[k] * 8);
      }
      if (!writes) {  // a flagged request: queries become 0, the cache stays
        if (b < 0 || kind || r.bad & SPECV_DEV_BAD_DRAFT_LEN) continue;
        w[0] = w[1] = make_uint4(0, 0, 0, 0);
      } else if (kind < 2 && (weight || half)) {
        float x[2][8];
#pragma unroll
        for (int k = 0; k < 2; k++)
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const float2 f = E::unpack((&w[k].x)[e]);
            x[k][2 * e] = f.x;
            x[k][2 * e + 1] = f.y;
          }
        if (weight) {
          float sum = 0.0f;
#pragma unroll
          for (int k = 0; k < 2; k++)
#pragma unroll
            for (int e = 0; e < 8; e++) sum = fmaf(x[k][e], x[k][e], sum);
#pragma unroll
          for (int o = kLanes / 2; o > 0; o /= 2) sum += __shfl_xor_sync(kFullMask, sum, o);
          const float inv = rsqrtf(sum / static_cast<float>(C.head_dim) + A.eps);
#pragma unroll
          for (int k = 0; k < 2; k++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const float2 f = E::unpack((&g[k].x)[e]);
              x[k][2 * e] = x[k][2 * e] * inv * f.x;
              x[k][2 * e + 1] = x[k][2 * e + 1] * inv * f.y;
            }
        }
        if (kOdd) {
          float* row = s_x[warp * kRowsAtOnce + group];
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 2; k++)
            if (mine[k]) {
              *reinterpret_cast<float4*>(row + piece[k] * 8) =
                  make_float4(x[k][0], x[k][1], x[k][2], x[k][3]);
              *reinterpret_cast<float4*>(row + piece[k] * 8 + 4) =
                  make_float4(x[k][4], x[k][5], x[k][6], x[k][7]);
            }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 2; k++)
#pragma unroll
            for (int e = 0; e < 8; e++) {
              const int d = piece[k] * 8 + e;
              if (!mine[k] || d >= A.rot_dim) continue;
              const float2 c = s_turn[warp][d < half ? d : d - half];
              x[k][e] = d < half ? x[k][e] * c.x - row[d + half] * c.y
                                 : x[k][e] * c.x + row[d - half] * c.y;
            }
        } else if (A.interleaved) {
          if (half)
#pragma unroll
            for (int k = 0; k < 2; k++)
#pragma unroll
              for (int e = 0; e < 4; e++) {
                const float a = x[k][2 * e], c = x[k][2 * e + 1];
                if (piece[k] * 4 + e < half) {
                  x[k][2 * e] = a * cs[k][e].x - c * cs[k][e].y;
                  x[k][2 * e + 1] = c * cs[k][e].x + a * cs[k][e].y;
                }
              }
        } else if (joined) {
#pragma unroll
          for (int e = 0; e < 8; e++) {
            const float2 f = cs[e / 4][e % 4];
            const float a = x[0][e], c = x[1][e];
            x[0][e] = a * f.x - c * f.y;
            x[1][e] = c * f.x + a * f.y;
          }
        }
#pragma unroll
        for (int k = 0; k < 2; k++)
#pragma unroll
          for (int e = 0; e < 4; e++) (&w[k].x)[e] = E::pack(x[k][2 * e], x[k][2 * e + 1]);
      }
      uint16_t* to = kind == 0 ? A.q_out.data + t * A.q_out.node_stride + h * A.q_out.head_stride
                               : (kind == 1 ? C.k : C.v) + slot + h * C.head_stride;
#pragma unroll
      for (int k = 0; k < 2; k++)
        if (mine[k] && h < (kind == 0 ? A.q_heads : C.heads))
          *reinterpret_cast<uint4*>(to + piece[k] * 8) = w[k];
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  for (int i = global; i < A.B; i += warps) {
    const unsigned bad = read_packed(P, i, call_bad, lane).bad;
    if (lane == 0) A.status[i] = static_cast<int32_t>(bad);
  }
}

template <class E>
void run_append_chunk(ChunkParams P, cudaStream_t stream) {
  const int half = P.a.rot_dim / 2;
  const bool odd = half % 8 != 0 && !P.a.interleaved, narrow = P.a.cache.head_dim <= 64;
  const int rows_at_once = narrow ? 8 : 4;
  const int passes = (P.a.q_heads + rows_at_once - 1) / rows_at_once +
                     2 * ((P.a.cache.heads + rows_at_once - 1) / rows_at_once);
  // As many warps as fit at a time; few tokens' heads are shared out over several.
  constexpr int kWarps = 3 * kAppendWarps * kSms;
  const int shares = P.T ? kWarps / P.T : 1;
  P.slices = shares < 1 ? 1 : shares < passes ? shares : passes;
  const int groups = kWarps / P.slices;  // of warps, a group to a token
  P.each = P.T / groups + (P.T % groups != 0);
  if (P.each < 1) P.each = 1;
  const int64_t warps = (static_cast<int64_t>(P.T) + P.each - 1) / P.each * P.slices;
  const int blocks = static_cast<int>((warps + kAppendWarps - 1) / kAppendWarps);
  const dim3 grid(blocks < 1 ? 1 : blocks);
  constexpr int kThreads = kAppendWarps * 32;
  if (narrow) {
    if (odd) append_chunk_kernel<E, 4, true><<<grid, kThreads, 0, stream>>>(P);
    else append_chunk_kernel<E, 4, false><<<grid, kThreads, 0, stream>>>(P);
  } else {
    if (odd) append_chunk_kernel<E, 8, true><<<grid, kThreads, 0, stream>>>(P);
    else append_chunk_kernel<E, 8, false><<<grid, kThreads, 0, stream>>>(P);
  }
}

// ------------------------------------------------------------------- keep

constexpr int kKeepThreads = 256;
constexpr int kBatch = 8;  // rows a thread has in flight

// A block's chain of loads (count, path, pages, rows) bounds it, three blocks of 66
// registers to an SM at a time: 128 requests, 16 layers, 8 + 8 heads of 128, up to 6 rows of
// each move in 16.4 us (50 MB, 3.1 TB/s), one layer of one request in 4.  (Several layers to a block, so that length and pages are read
// less often, took 15.9 to 16.5 us; more warps to an SM, of fewer registers, 23 to 30.)
//
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
                       B,
                       N,
                       q_heads,
                       rot_dim,
                       interleaved};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (cache->dtype == SPECV_BF16) run_append<Bf16>(P, st);
  else run_append<F16>(P, st);
  return launched();
}

specv_status spec_append_chunk(const specv_cache* cache, const specv_rows* q, const specv_rows* k,
                               const specv_rows* v, const int32_t* cu_tokens, int B, int T,
                               int q_heads, const int32_t* positions, int64_t position_stride,
                               int axes, const int32_t* axis_of, const void* q_weight,
                               const void* k_weight, float eps, const float* inv_freq, int rot_dim,
                               int interleaved, float rope_scale, const specv_rows* q_out,
                               int32_t* status, specv_stream_t stream) {
  const specv_status s = check_cache(cache, B, 1);
  if (s != SPECV_OK) return s;
  if (!rows_ok(q) || !rows_ok(k) || !rows_ok(v) || !rows_ok(q_out) || !cu_tokens || !status ||
      q_heads < 1 || T < 0 || rot_dim < 0 || rot_dim % 2 != 0 || rot_dim > cache->head_dim ||
      (rot_dim > 0) != !!inv_freq || cache->layers != 1)
    return SPECV_ERR_INVALID_ARG;
  if (positions ? axes < 1 || position_stride < 0 || (axes > 1 && (position_stride < T || !axis_of))
                : axis_of || axes > 1)
    return SPECV_ERR_INVALID_ARG;
  if (!aligned_to(cu_tokens, 4) || !aligned_to(positions, 4) || !aligned_to(axis_of, 4) ||
      !aligned_to(q_weight, 16) || !aligned_to(k_weight, 16) || !aligned_to(inv_freq, 4) ||
      !aligned_to(status, 4))
    return SPECV_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || eps > 3e38f || !(rope_scale > -3e38f && rope_scale < 3e38f))
    return SPECV_ERR_INVALID_ARG;
  if (q_heads > 1024) return SPECV_ERR_UNSUPPORTED;
  const ChunkParams P{{to_cache(cache),
                       to_rows(q),
                       to_rows(k),
                       to_rows(v),
                       to_rows(q_out),
                       nullptr,
                       nullptr,
                       static_cast<const uint16_t*>(q_weight),
                       static_cast<const uint16_t*>(k_weight),
                       inv_freq,
                       status,
                       eps,
                       rope_scale,
                       B,
                       1,
                       q_heads,
                       rot_dim,
                       interleaved},
                      cu_tokens,
                      positions,
                      axis_of,
                      position_stride,
                      T,
                      axes,
                      1,
                      1};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (cache->dtype == SPECV_BF16) run_append_chunk<Bf16>(P, st);
  else run_append_chunk<F16>(P, st);
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
