// Attention of single tokens over the paged cache: a call in which no request has
// more than one, and a key head has up to 16 query heads.
//
// All rows of a key head see the same slots, so there are no masks, and the work is the
// keys' and values' bytes.  A cluster of CTAs has a request's key head and shares out
// its slots, 64 to a warp at a time: S = Q K^T by warp-wide MMAs with the keys' fragments
// loaded from the cache as they lie (a row's columns are summed in an order that gives each
// lane 16 bytes of it), the weights passed on as fragments, values through shared memory.
// The warps' (m, l, O) are joined in their CTA, the CTAs' through the cluster's
// shared memory: one kernel.
//
// For few bytes, where a call is latencies and the fetching of code: one request of 32 + 8 heads
// of 128, a slot 10.4 us (tiles of 128 rows and a second kernel for the join: 14.7), 4,002 slots
// 12.4 (20), 32,002 slots 67 (42); 16 requests of 2,000 to 6,000 slots 88 to 99 (62).
#pragma once

#include "chunk.cuh"

namespace specv_chunk {

constexpr int kOneRows = 16;    // rows of an MMA's tile
constexpr int kOneWarps = 8;
constexpr int kOneKeys = 64;    // slots of a warp at a time
constexpr int kMostCtas = 8;    // of a cluster

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                         Bf16) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                         F16) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four 8 x 8 matrices of 16 bits, transposed; this lane's row of one of them is at `at`.
__device__ __forceinline__ void load_transposed(uint32_t at, uint32_t (&x)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
               : "r"(at)
               : "memory");
}

__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A number in the shared memory of the cluster's CTA `rank`, at this CTA's address `at`.
__device__ __forceinline__ float cluster_load(uint32_t at, int rank) {
  uint32_t there;
  float x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(there) : "memory");
  return x;
}

// What the warps, and then the CTAs, leave for one another.
template <int DP> struct OneTail {
  float o[kOneWarps][kOneRows][DP];  // over the values, when all have been read
};
struct OneStats {
  float m[kOneWarps][kOneRows], l[kOneWarps][kOneRows];
  float m_all[kOneRows], l_all[kOneRows];
  int bad;
};

// grid: (cluster's CTAs, key heads, requests)
template <class E, int DP>
__global__ void __launch_bounds__(kOneWarps * 32, 1) single_kernel(const Params P) {
  constexpr int kPieces = DP / 8;   // 16-byte pieces of a row
  constexpr int kVectors = DP / 32; // of them a lane has
  extern __shared__ __align__(1024) char smem[];
  OneStats& s = *reinterpret_cast<OneStats*>(smem + kOneWarps * kOneKeys * DP * 2);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, quad = lane & 3, group = lane / 4;
  const int b = blockIdx.z, h = blockIdx.y, rank = blockIdx.x, ctas = gridDim.x;
  const Cache& C = P.cache;
  const Request r = request_of(P, b);
  const int pieces = C.head_dim / 8;
  if (tid == 0) s.bad = 0;
  __syncthreads();

  // The slots that the token sees, in their order: the prefix's, then the window's.
  const int pos = r.len, low = lowest(P, pos);
  const int own = min(r.prefix, low);
  const int count = r.bad || r.n != 1 ? 0 : own + pos + 1 - low;
  auto slot_of = [&](int i) { return i < own ? i : low + i - own; };
  const int32_t* table = C.page_table + static_cast<int64_t>(b) * C.table_stride;

  // Queries as fragments: rows `group` and `group` + 8, where a lane's 16 bytes of 32 columns
  // are what two steps of 16 take from it.
  uint32_t q[2 * kVectors][4];
#pragma unroll
  for (int j = 0; j < kVectors; j++) {
    uint4 w[2];
#pragma unroll
    for (int k = 0; k < 2; k++) {
      const int row = group + 8 * k, piece = 4 * j + quad;
      w[k] = make_uint4(0, 0, 0, 0);
      if (count && row < P.group && piece < pieces)
        w[k] = *reinterpret_cast<const uint4*>(P.q.data + r.first * P.q.node_stride +
                                               (h * P.group + row) * P.q.head_stride + piece * 8);
    }
#pragma unroll
    for (int t = 0; t < 2; t++) {
      q[2 * j + t][0] = t ? w[0].z : w[0].x;
      q[2 * j + t][1] = t ? w[1].z : w[1].x;
      q[2 * j + t][2] = t ? w[0].w : w[0].y;
      q[2 * j + t][3] = t ? w[1].w : w[1].y;
    }
  }
  float slope[2] = {0.0f, 0.0f};
  if (P.slopes && count)
#pragma unroll
    for (int k = 0; k < 2; k++)
      if (group + 8 * k < P.group) slope[k] = P.slopes[h * P.group + group + 8 * k] * 1.4426950408889634f;

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};  // l: of this lane's columns
  float o[kPieces][4];
#pragma unroll
  for (int n = 0; n < kPieces; n++)
#pragma unroll
    for (int e = 0; e < 4; e++) o[n][e] = 0.0f;
  char* const values = smem + warp * kOneKeys * DP * 2;
  const uint32_t values_at = smem_of(values);

#pragma unroll 1
  for (int first = (rank * kOneWarps + warp) * kOneKeys; first < count; first += ctas * kOneWarps * kOneKeys) {
    // Offsets of this lane's two slots, -1 where there is none (or no such page: the request is
    // flagged below).
    int64_t at[2];
#pragma unroll
    for (int k = 0; k < 2; k++) {
      const int i = first + 32 * k + lane;
      at[k] = -1;
      if (i < count) {
        const int slot = slot_of(i), page = table[slot / C.page_size];
        if (page >= 0 && page < C.pages)
          at[k] = page * C.page_stride + slot % C.page_size * C.row_stride + h * C.head_stride;
      }
    }
    auto offset = [&](int i) { return __shfl_sync(kFullMask, i < 32 ? at[0] : at[1], i & 31); };
    // The values of all 64, pieces swapped by the slot's number
    __syncwarp();
#pragma unroll 4
    for (int e = lane; e < kOneKeys * kPieces; e += 32) {
      const int i = e / kPieces, piece = e % kPieces;
      // (32 / kPieces slots at a time, so all lanes ask for the same half's offsets)
      const int64_t off = offset(i);
      const bool real = off >= 0 && piece < pieces;
      copy16(values_at + i * (DP * 2) + (piece ^ (i & 7)) * 16, C.v + (real ? off + piece * 8 : 0), real);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    // Scores, 32 slots at a time: slot 8 n + group of a lane's keys
    float x[kOneKeys / 8][4];
#pragma unroll
    for (int part = 0; part < 2; part++) {
      uint4 k[4][kVectors];
#pragma unroll
      for (int n = 0; n < 4; n++) {
        const int64_t off = offset(32 * part + 8 * n + group);
#pragma unroll
        for (int j = 0; j < kVectors; j++) {
          k[n][j] = make_uint4(0, 0, 0, 0);
          if (off >= 0 && 4 * j + quad < pieces)
            k[n][j] = *reinterpret_cast<const uint4*>(C.k + off + (4 * j + quad) * 8);
        }
      }
#pragma unroll
      for (int n = 0; n < 4; n++) {
        float (&d)[4] = x[4 * part + n];
#pragma unroll
        for (int e = 0; e < 4; e++) d[e] = 0.0f;
#pragma unroll
        for (int j = 0; j < kVectors; j++) {
          mma16816(d, q[2 * j], k[n][j].x, k[n][j].y, E());
          mma16816(d, q[2 * j + 1], k[n][j].z, k[n][j].w, E());
        }
      }
    }
    // x[n][2 k + e]: row group + 8 k, slot 8 n + 2 quad + e
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < kOneKeys / 8; n++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
        const int i = first + 8 * n + 2 * quad + e;
        const float away = static_cast<float>(pos - slot_of(i));
#pragma unroll
        for (int k = 0; k < 2; k++) {
          float y = x[n][2 * k + e];
          y = P.cap_log2 > 0.0f ? capped(P, y) : y * P.scale_log2;
          y = fmaf(-slope[k], away, y);
          if (i >= count) y = -INFINITY;
          x[n][2 * k + e] = y;
          top[k] = fmaxf(top[k], y);
        }
      }
    float by[2];
#pragma unroll
    for (int k = 0; k < 2; k++) {
#pragma unroll
      for (int f = 1; f < 4; f *= 2) top[k] = fmaxf(top[k], __shfl_xor_sync(kFullMask, top[k], f));
      const float higher = fmaxf(m[k], top[k]);
      by[k] = m[k] == higher ? 1.0f : exp2_of(m[k] - higher);
      m[k] = higher;
      l[k] *= by[k];
    }
#pragma unroll
    for (int n = 0; n < kPieces; n++)
#pragma unroll
      for (int e = 0; e < 4; e++) o[n][e] *= by[e / 2];
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    // (weights in f16 are taken 2^7 larger, so that fewer are below 2^-14, where its steps stop
    // shrinking)
    constexpr float kLift = std::is_same<E, F16>::value ? 7.0f : 0.0f;
    const float shift[2] = {kLift - (m[0] == -INFINITY ? 0.0f : m[0]), kLift - (m[1] == -INFINITY ? 0.0f : m[1])};
#pragma unroll
    for (int step = 0; step < kOneKeys / 16; step++) {
      uint32_t p[4];
#pragma unroll
      for (int half = 0; half < 2; half++)
#pragma unroll
        for (int k = 0; k < 2; k++) {
          const float* y = x[2 * step + half] + 2 * k;
          const float a = exp2_of(y[0] + shift[k]), c = exp2_of(y[1] + shift[k]);
          l[k] += a + c;
          // the weights' one rounding, to the type of the values they meet
          p[2 * half + k] = E::pack(a, c);
        }
#pragma unroll
      for (int n = 0; n < kPieces; n += 2) {
        // keys 16 step + 0..7 and 8..15 of columns 8 n .. 8 n + 7, then of the next eight
        const int i = 16 * step + (lane & 15), piece = n + lane / 16;
        uint32_t v[4];
        load_transposed(values_at + i * (DP * 2) + (piece ^ (i & 7)) * 16, v);
        mma16816(o[n], p, v[0], v[1], E());
        mma16816(o[n + 1], p, v[2], v[3], E());
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 2; k++)
#pragma unroll
    for (int f = 1; f < 4; f *= 2) l[k] += __shfl_xor_sync(kFullMask, l[k], f);

  // This warp's share of the pages' check: those of slots that the token sees.
  if (count) {
    const bool bad = bad_pages(C, b, 0, own, tid, kOneWarps * 32) ||
                     bad_pages(C, b, low, pos + 1, tid, kOneWarps * 32);
    if (bad) s.bad = 1;
  }
  __syncthreads();  // all values have been read
  OneTail<DP>& tail = *reinterpret_cast<OneTail<DP>*>(smem);
#pragma unroll
  for (int k = 0; k < 2; k++) {
    const int row = group + 8 * k;
    if (quad == 0) {
      s.m[warp][row] = m[k];
      s.l[warp][row] = l[k];
    }
    if (row < P.group)
#pragma unroll
      for (int n = 0; n < kPieces; n++)
        *reinterpret_cast<float2*>(&tail.o[warp][row][8 * n + 2 * quad]) = make_float2(o[n][2 * k], o[n][2 * k + 1]);
  }
  __syncthreads();
  // The CTA's rows, into the first warp's place
  const int all = P.group * DP;
  for (int e = tid; e < all; e += kOneWarps * 32) {
    const int row = e / DP, d = e % DP;
    float top = -INFINITY, sum = 0.0f, total = 0.0f;
#pragma unroll
    for (int w = 0; w < kOneWarps; w++) top = fmaxf(top, s.m[w][row]);
#pragma unroll
    for (int w = 0; w < kOneWarps; w++) {
      const float weight = s.m[w][row] == top ? 1.0f : exp2_of(s.m[w][row] - top);
      total = fmaf(weight, s.l[w][row], total);
      sum = fmaf(weight, tail.o[w][row][d], sum);
    }
    tail.o[0][row][d] = sum;  // (no other thread's)
    if (d == 0) {
      s.m_all[row] = top;
      s.l_all[row] = total;
    }
  }
  cluster_barrier();
  // The cluster's rows, shared out over its CTAs
  const bool flagged = r.bad || s.bad;  // every CTA has looked at all pages
  uint16_t* const out = P.out.data + r.first * P.out.node_stride + static_cast<int64_t>(h) * P.group * P.out.head_stride;
  if (count)
    for (int e = 2 * (rank * kOneWarps * 32 + tid); e < all; e += 2 * ctas * kOneWarps * 32) {
      const int row = e / DP, d = e % DP;
      if (d >= C.head_dim) continue;
      float ms[kMostCtas], top = -INFINITY, total = 0.0f, sum[2] = {0.0f, 0.0f};
      for (int c = 0; c < ctas; c++) top = fmaxf(top, ms[c & 7] = cluster_load(smem_of(&s.m_all[row]), c));
      for (int c = 0; c < ctas; c++) {
        const float weight = ms[c & 7] == top ? 1.0f : exp2_of(ms[c & 7] - top);
        total = fmaf(weight, cluster_load(smem_of(&s.l_all[row]), c), total);
        sum[0] = fmaf(weight, cluster_load(smem_of(&tail.o[0][row][d]), c), sum[0]);
        sum[1] = fmaf(weight, cluster_load(smem_of(&tail.o[0][row][d + 1]), c), sum[1]);
      }
      const float inv = 1.0f / total;
      *reinterpret_cast<uint32_t*>(out + row * P.out.head_stride + d) =
          flagged ? 0u : E::pack(sum[0] * inv, sum[1] * inv);
    }
  if (rank == 0 && h == 0 && tid == 0) P.status[b] = static_cast<int32_t>(r.bad | (s.bad ? SPECV_DEV_BAD_CACHE : 0));
  // A request that was refused before its rows were looked at: they become 0.
  if (r.bad && rank == 0) {
    const int64_t words = static_cast<int64_t>(r.n) * P.group * pieces;
    for (int64_t e = tid; e < words; e += kOneWarps * 32) {
      const int64_t i = e / (P.group * pieces);
      const int left = static_cast<int>(e - i * (P.group * pieces)), row = left / pieces, piece = left % pieces;
      *reinterpret_cast<uint4*>(P.out.data + (r.first + i) * P.out.node_stride +
                                (h * P.group + row) * P.out.head_stride + piece * 8) = make_uint4(0, 0, 0, 0);
    }
  }
  cluster_barrier();  // no CTA leaves while another reads from it
}

template <class E, int DP>
cudaError_t launch_single(const Params& P, cudaStream_t stream) {
  constexpr int kValues = kOneWarps * kOneKeys * DP * 2;
  static_assert(sizeof(OneTail<DP>) <= kValues, "the joined rows lie where the values were");
  constexpr int kSmem = kValues + static_cast<int>(sizeof(OneStats));
  const cudaError_t e = cudaFuncSetAttribute(single_kernel<E, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  int ctas = kMostCtas;
  while (ctas > 1 && P.B * P.cache.heads * ctas > kSms) ctas /= 2;  // one to an SM
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {static_cast<unsigned>(ctas), 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, P.cache.heads, P.B);
  cfg.blockDim = dim3(kOneWarps * 32);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, single_kernel<E, DP>, P);
}

}  // namespace specv_chunk
