// The drafting of a tree, or a beam search's step: the best of all beams' next
// tokens, and their states moved along.
//
//   score(w, v) = scores[w] + z[w,v] - log sum_u exp z[w,u],
//
// the K best of W V.  Within a row the order is that of z, so a block that has a part of a
// row keeps that part's K best entries and its max and sum of exponentials; a request's
// block then has the rows' sums, turns the W parts' entries into scores and takes the K
// best of them.  Each logit is read once, and only the few that may be among the best
// leave the registers.

#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "cache.cuh"

using namespace specv_cache_ops;

namespace {

constexpr int kThreads = 256;
constexpr int kMine = 32;                  // entries of a tile that a thread has
constexpr int kTile = kThreads * kMine;    // entries of a row that a block looks at together
constexpr int kMaxBeams = SPECV_MAX_BEAMS;
constexpr int kFound = 1024;  // entries that may be among the best, of a tile or of a request
constexpr int kVocabBits = 20;  // of a vocabulary entry's number

template <int DT> struct Elt;
template <> struct Elt<SPECV_F32> {
  using T = float;
  static constexpr int kVec = 4;
  static __device__ __forceinline__ float one(float x) { return x; }
  static __device__ __forceinline__ void unpack(const uint4& v, float* z) {
    z[0] = __uint_as_float(v.x);
    z[1] = __uint_as_float(v.y);
    z[2] = __uint_as_float(v.z);
    z[3] = __uint_as_float(v.w);
  }
};
template <> struct Elt<SPECV_BF16> {
  using T = uint16_t;
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float one(uint16_t x) {
    return __uint_as_float(static_cast<uint32_t>(x) << 16);
  }
  static __device__ __forceinline__ void unpack(const uint4& v, float* z) {
    const uint32_t* w = &v.x;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      z[2 * i] = __uint_as_float(w[i] << 16);
      z[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

// What a block leaves of its part of a row; behind it K keys, best first, 0: none.
struct Part {
  float max;
  float pad;
  double sum;  // of exp(z - max)
};

struct Params {
  const void* logits;
  int64_t batch_stride, row_stride;  // elements
  const float* scores;
  const int32_t* ended;
  Part* parts;      // [B W, splits]
  uint64_t* keys;   // [B W, splits, K]
  float* out_scores;
  int32_t* tokens;
  int32_t* beams;
  int32_t* status;
  int W, V, K, splits, tiles, end_token;  // tiles: of a part
};

// An entry of a row as one number: a larger value, then a smaller place, is larger.
__device__ __forceinline__ uint64_t key_of(float z, int at) {
  const uint32_t u = __float_as_uint(z + 0.0f);  // (-0 is 0)
  const uint32_t ordered = u >> 31 ? ~u : u | 0x80000000u;
  return static_cast<uint64_t>(ordered) << 32 | (0xffffffffu - static_cast<uint32_t>(at));
}
__device__ __forceinline__ float value_of(uint64_t key) {
  const uint32_t u = static_cast<uint32_t>(key >> 32);
  return __uint_as_float(u >> 31 ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ int place_of(uint64_t key) {
  return static_cast<int>(0xffffffffu - static_cast<uint32_t>(key));
}

__device__ __forceinline__ float exp_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}

// The vector of a row's entries from `at` on.  A row may begin anywhere: then two
// aligned vectors are shifted together where both lie within the row.
template <int DT>
__device__ __forceinline__ void load_vector(const typename Elt<DT>::T* row, int at, int V, int shift,
                                            float* z) {
  using E = Elt<DT>;
  constexpr int kVec = E::kVec, kSize = 16 / kVec;
  if (at + kVec <= V && shift == 0) {
    E::unpack(__ldg(reinterpret_cast<const uint4*>(row + at)), z);
  } else if (at * kSize >= shift && (at + 2 * kVec) * kSize - shift <= V * static_cast<int64_t>(kSize)) {
    const uint4* from = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(row + at) - shift);
    const uint4 a = __ldg(from), b = __ldg(from + 1);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t x[5];
    const int words = shift / 4;
#pragma unroll
    for (int i = 0; i < 5; i++)
      x[i] = words == 0 ? w[i] : words == 1 ? w[i + 1] : words == 2 ? w[i + 2] : w[i + 3];
    uint4 v;
#pragma unroll
    for (int i = 0; i < 4; i++) (&v.x)[i] = shift % 4 ? __funnelshift_r(x[i], x[i + 1], 16) : x[i];
    E::unpack(v, z);
  } else {
#pragma unroll
    for (int i = 0; i < kVec; i++) z[i] = at + i < V ? E::one(row[at + i]) : -INFINITY;
  }
}

// A block's part of one row.
template <int DT>
__global__ void __launch_bounds__(kThreads, 4) select_rows_kernel(const Params P) {
  using E = Elt<DT>;
  constexpr int kVec = E::kVec;
  __shared__ uint64_t s_found[kFound];
  __shared__ uint64_t s_best[2][kMaxBeams];
  __shared__ float s_top[kMaxBeams];
  __shared__ float s_max[kThreads / 32];
  __shared__ double s_sum[kThreads / 32];
  __shared__ int s_count[3];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  const int64_t row = blockIdx.x / P.splits;
  const int split = blockIdx.x - static_cast<int>(row) * P.splits, K = P.K;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // A beam that has ended or is not in play has no row.
  if (P.scores[row] == -INFINITY || (P.ended && P.ended[row])) return;
  const auto* from = static_cast<const typename E::T*>(P.logits) + row / P.W * P.batch_stride +
                     row % P.W * P.row_stride;
  const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(from) & 15);

  float m = -INFINITY;
  double l = 0.0;
  int have = 0, now = 0;  // entries of s_best[now]
  // groups of threads, at least K of them: each has an entry of its own maximum
  const int groups = K <= 8 ? 8 : K <= 16 ? 16 : K <= 32 ? 32 : 64, width = kThreads / groups;
  for (int tile = 0; tile < P.tiles; tile++) {
    const int first = (split * P.tiles + tile) * kTile;
    if (first >= P.V) break;
    float z[kMine];
#pragma unroll
    for (int j = 0; j < kMine / kVec; j++)
      load_vector<DT>(from, first + (j * kThreads + tid) * kVec, P.V, shift, z + j * kVec);
    float top = z[0];
#pragma unroll
    for (int j = 1; j < kMine; j++) top = fmaxf(top, z[j]);
    const float higher = fmaxf(m, top);
    float sum = 0.0f;
    // (a row of a NaN or +inf makes the sum a NaN, which the request's block sees)
#pragma unroll
    for (int j = 0; j < kMine; j++) sum += exp_of(z[j] - (higher == -INFINITY ? 0.0f : higher));
    l = l * (higher == -INFINITY ? 1.0 : static_cast<double>(exp_of(m - higher))) + sum;
    m = higher;

    if (tid < 3) s_count[tid] = 0;
    float least;  // an entry below it is not among the K best
    if (tile == 0) {
      float all = top;
      for (int o = width / 2; o > 0; o /= 2) all = fmaxf(all, __shfl_xor_sync(kFullMask, all, o));
      if (tid % width == 0) s_top[tid / width] = all;
      __syncthreads();
      least = s_top[0];
      for (int g = 1; g < groups; g++) least = fminf(least, s_top[g]);
    } else {
      __syncthreads();
      least = have < K ? -INFINITY : value_of(s_best[now][K - 1]);
    }
    // (behind the first tile a value equal to the K-th comes later than it)
    const bool equal = tile == 0 && least > -INFINITY;
    if (equal ? top >= least : top > least) {
#pragma unroll
      for (int j = 0; j < kMine; j++)
        if (equal ? z[j] >= least : z[j] > least) {
          const int at = atomicAdd(&s_count[0], 1);
          if (at < kFound)
            s_found[at] = key_of(z[j], first + (j / kVec * kThreads + tid) * kVec + j % kVec);
        }
    }
    __syncthreads();
    int found = s_count[0];
    if (found > kFound) {
      // Too many: the tile's K-th best itself, bit by bit from the top of its value and place.
      constexpr int kBits = 32 + kVocabBits;
      auto small_key = [&](int j) {
        const int at = first + (j / kVec * kThreads + tid) * kVec + j % kVec;
        return z[j] > -INFINITY ? key_of(z[j], at) >> 32 << kVocabBits | ((1 << kVocabBits) - 1 - at) : 0ull;
      };
      uint64_t least_key = 0;
      for (int bit = kBits - 1; bit >= 0; bit--) {
        const uint64_t at_least = least_key | 1ull << bit;
        int n = 0;
#pragma unroll
        for (int j = 0; j < kMine; j++) n += small_key(j) >= at_least;
        n = __reduce_add_sync(kFullMask, n);
        int* count = &s_count[1 + bit % 2];
        if (lane == 0 && n) atomicAdd(count, n);
        __syncthreads();
        if (*count >= K) least_key = at_least;
        if (tid == 0) s_count[1 + (bit + 1) % 2] = 0;
        __syncthreads();
      }
      if (tid == 0) s_count[0] = 0;
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kMine; j++)
        if (small_key(j) >= least_key && z[j] > -INFINITY)
          s_found[atomicAdd(&s_count[0], 1)] =
              key_of(z[j], first + (j / kVec * kThreads + tid) * kVec + j % kVec);
      __syncthreads();
      found = s_count[0];
    }
    if (found) {
      // The best of those so far and the found, each at the place that its rank is.
      auto nth = [&](int i) { return i < have ? s_best[now][i] : s_found[i - have]; };
      const int all = have + found;
      for (int i = tid; i < all; i += kThreads) {
        const uint64_t key = nth(i);
        int rank = 0;
        for (int k = 0; k < have; k++) rank += s_best[now][k] > key;
        for (int k = 0; k < found; k++) rank += s_found[k] > key;
        if (rank < K) s_best[now ^ 1][rank] = key;
      }
      have = min(K, all);
      now ^= 1;
    }
    __syncthreads();
  }
  // The part's maximum and sum.
  float all = m;
#pragma unroll
  for (int o = 16; o > 0; o /= 2) all = fmaxf(all, __shfl_xor_sync(kFullMask, all, o));
  if (lane == 0) s_max[warp] = all;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; w++) all = fmaxf(all, s_max[w]);
  if (all > -INFINITY) l *= static_cast<double>(exp_of(m - all));
#pragma unroll
  for (int o = 16; o > 0; o /= 2) l += __shfl_xor_sync(kFullMask, l, o);
  if (lane == 0) s_sum[warp] = l;
  __syncthreads();
  const int64_t at = row * P.splits + split;
  if (tid == 0) {
    double sum = 0.0;
    for (int w = 0; w < kThreads / 32; w++) sum += s_sum[w];
    P.parts[at] = Part{all, 0.0f, sum};
  }
  if (tid < K) P.keys[at * K + tid] = tid < have ? s_best[now][tid] : 0;
}

// A candidate: its score, and beam and token as one number.
struct Candidate {
  double score;
  uint32_t place;
};
__device__ __forceinline__ bool better(const Candidate& a, const Candidate& b) {
  return a.score > b.score || (a.score == b.score && a.place < b.place);
}
__device__ __forceinline__ Candidate best_of_warp(Candidate c, int width) {
  for (int o = width / 2; o > 0; o /= 2) {
    const Candidate d{__shfl_xor_sync(kFullMask, c.score, o), __shfl_xor_sync(kFullMask, c.place, o)};
    if (better(d, c)) c = d;
  }
  return c;
}

// A request's block: the rows' sums, then the K best of the parts' entries.
__global__ void __launch_bounds__(kThreads) select_kernel(const Params P) {
  __shared__ double s_off[kMaxBeams];  // score - log sum of a row; an ended beam's score
  __shared__ float s_max[kMaxBeams];   // and what that sum's exponentials were taken from
  __shared__ uint8_t s_kind[kMaxBeams];  // 0: no candidate, 1: a row, 2: ended
  __shared__ Candidate s_found[kFound];
  __shared__ double s_top[kMaxBeams];
  __shared__ Candidate s_warp[kThreads / 32];
  __shared__ int s_count, s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  const int64_t b = blockIdx.x;
  const int W = P.W, K = P.K;
  if (tid == 0) s_count = s_bad = 0;
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int w = warp; w < W; w += kThreads / 32) {
    const int64_t row = b * W + w;
    const float score = P.scores[row];
    const bool over = P.ended && P.ended[row];
    unsigned bad = 0;
    if (!(score < INFINITY)) bad = SPECV_DEV_BAD_BEAM;
    double off = score;
    int kind = score == -INFINITY || bad ? 0 : over ? 2 : 1;
    if (kind == 1) {
      float m = -INFINITY;
      for (int k = lane; k < P.splits; k += 32) m = fmaxf(m, P.parts[row * P.splits + k].max);
#pragma unroll
      for (int o = 16; o > 0; o /= 2) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, o));
      double sum = 0.0;
      for (int k = lane; k < P.splits; k += 32) {
        const Part part = P.parts[row * P.splits + k];
        // (a part of -inf alone has 0, one that has a NaN a NaN)
        sum += part.max == -INFINITY
                   ? part.sum * 0.0
                   : part.sum * exp(static_cast<double>(part.max) - static_cast<double>(m));
      }
#pragma unroll
      for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(kFullMask, sum, o);
      if (sum != sum || m == INFINITY) bad = SPECV_DEV_BAD_ROW, kind = 0;
      else if (m == -INFINITY) kind = 0;  // nothing is allowed
      else off = static_cast<double>(score) - log(sum);
      if (lane == 0) s_max[w] = m;
    }
    if (lane == 0) {
      s_off[w] = off;
      s_kind[w] = static_cast<uint8_t>(kind);
      if (bad) atomicOr(&s_bad, static_cast<int>(bad));
    }
  }
  __syncthreads();
  const int per_row = P.splits * K, all = W * per_row;
  // Entry number e; worse than any where there is none.
  const Candidate none{-INFINITY, 0xffffffffu};
  auto entry = [&](int e) {
    const int w = e / per_row, k = e - w * per_row, kind = s_kind[w];
    if (kind == 0 || (kind == 2 && k)) return none;
    const uint32_t beam = static_cast<uint32_t>(w) << kVocabBits;
    if (kind == 2) return Candidate{s_off[w], beam};
    const uint64_t key = P.keys[(b * W + w) * per_row + k];
    if (!key) return none;
    return Candidate{s_off[w] + (static_cast<double>(value_of(key)) - static_cast<double>(s_max[w])),
                     beam | static_cast<uint32_t>(place_of(key))};
  };
  const bool bad = s_bad != 0;
  // The least of K or more groups' best: nothing below it is among the K best.
  double mine = -INFINITY;
  if (!bad)
    for (int e = tid; e < all; e += kThreads) mine = fmax(mine, entry(e).score);
  const int groups = K <= 8 ? 8 : K <= 16 ? 16 : K <= 32 ? 32 : 64, width = kThreads / groups;
  for (int o = width / 2; o > 0; o /= 2) mine = fmax(mine, __shfl_xor_sync(kFullMask, mine, o));
  if (tid % width == 0) s_top[tid / width] = mine;
  __syncthreads();
  double least = s_top[0];
  for (int g = 1; g < groups; g++) least = fmin(least, s_top[g]);
  if (!bad)
    for (int e = tid; e < all; e += kThreads) {
      const Candidate c = entry(e);
      if (c.score > -INFINITY && c.score >= least) {
        const int at = atomicAdd(&s_count, 1);
        if (at < kFound) s_found[at] = c;
      }
    }
  __syncthreads();
  const int found = s_count;
  auto put = [&](int k, const Candidate& c) {
    const bool real = c.score > -INFINITY;
    const int w = static_cast<int>(c.place >> kVocabBits);
    P.out_scores[b * K + k] = static_cast<float>(c.score);
    P.beams[b * K + k] = real ? w : -1;
    P.tokens[b * K + k] = !real ? -1 : s_kind[w] == 2 ? P.end_token
                                                      : static_cast<int>(c.place & ((1u << kVocabBits) - 1));
  };
  if (found <= kFound) {
    for (int i = tid; i < found; i += kThreads) {
      const Candidate c = s_found[i];
      int rank = 0;
      for (int k = 0; k < found; k++) rank += better(s_found[k], c);
      if (rank < K) put(rank, c);
    }
    for (int k = found + tid; k < K; k += kThreads) put(k, none);
  } else {
    // Too many (scores all alike): one after the other, each the best of those behind the last.
    Candidate last{INFINITY, 0};
    for (int k = 0; k < K; k++) {
      Candidate c = none;
      for (int e = tid; e < all; e += kThreads) {
        const Candidate d = entry(e);
        if (better(last, d) && better(d, c)) c = d;
      }
      c = best_of_warp(c, 32);
      if (lane == 0) s_warp[warp] = c;
      __syncthreads();
      c = s_warp[0];
      for (int i = 1; i < kThreads / 32; i++)
        if (better(s_warp[i], c)) c = s_warp[i];
      __syncthreads();
      if (tid == 0) put(k, c);
      last = c;
    }
  }
  if (tid == 0) P.status[b] = s_bad;
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// How rows are shared out over blocks, and the workspace for it.
struct Plan {
  int tiles, splits;  // of a part, of a row
  size_t keys, total;

  Plan(int B, int W, int K, int V) {
    const int all = (V + kTile - 1) / kTile;
    const int64_t rows = static_cast<int64_t>(B) * W, wanted = 16 * kSms;
    const int parts = static_cast<int>(rows >= wanted ? 1 : (wanted + rows - 1) / rows);
    tiles = parts >= all ? 1 : (all + parts - 1) / parts;
    splits = (all + tiles - 1) / tiles;
    keys = align256(rows * splits * sizeof(Part));
    total = keys + align256(rows * splits * K * sizeof(uint64_t));
  }
};

specv_status check_beams(int B, int W, int K) {
  if (B < 1 || W < 1 || K < 1) return SPECV_ERR_INVALID_ARG;
  return B > SPECV_MAX_BATCH || W > kMaxBeams || K > kMaxBeams ? SPECV_ERR_UNSUPPORTED : SPECV_OK;
}

// ----------------------------------------------------------------- reorder

constexpr int kMoveThreads = 128;

struct Moved {
  const char* in;
  char* out;
  int64_t in_batch, in_beam, out_batch, out_beam, bytes;
  int unit;        // bytes that a thread moves of a row
  int first_tile;  // of all states' columns
};

struct MoveParams {
  const int32_t* beams;
  int32_t* status;
  int W, K, states;
  Moved state[SPECV_MAX_STATES];
};

// Moves this thread's column of a state: all its loads before its first store, so that a
// state may be moved within itself.
template <class T, int kMost>
__device__ __forceinline__ void move_column(const Moved& s, int64_t b, int64_t at, const int* beams, int K) {
  const char* in = s.in + b * s.in_batch + at;
  char* out = s.out + b * s.out_batch + at;
  T x[kMost];
#pragma unroll
  for (int k = 0; k < kMost; k++)
    if (k < K && beams[k] >= 0) x[k] = *reinterpret_cast<const T*>(in + beams[k] * s.in_beam);
#pragma unroll
  for (int k = 0; k < kMost; k++)
    if (k < K && beams[k] >= 0) *reinterpret_cast<T*>(out + k * s.out_beam) = x[k];
}

// A block has a request and a run of columns of one state, a thread one of them in every beam.
template <int kMost>
__global__ void __launch_bounds__(kMoveThreads) reorder_kernel(const __grid_constant__ MoveParams P) {
  __shared__ int s_beams[kMaxBeams];
  const int tid = threadIdx.x;
  const int64_t b = blockIdx.y + static_cast<int64_t>(blockIdx.z) * 32768;
  bool bad = false;
  if (tid < P.K) {
    const int w = P.beams[b * P.K + tid];
    s_beams[tid] = w;
    bad = w < -1 || w >= P.W;
  }
  bad = __syncthreads_or(bad);
  const int tile = blockIdx.x;
  if (tile == 0 && tid == 0) P.status[b] = bad ? SPECV_DEV_BAD_BEAM : 0;
  if (bad) return;
  int i = 0;
  while (i + 1 < P.states && tile >= P.state[i + 1].first_tile) i++;
  const Moved& s = P.state[i];
  const int64_t at = (static_cast<int64_t>(tile - s.first_tile) * kMoveThreads + tid) * s.unit;
  if (at >= s.bytes) return;
  if (kMost <= 16 && s.unit == 16) move_column<uint4, kMost>(s, b, at, s_beams, P.K);
  else if (kMost <= 32 && s.unit == 8) move_column<uint2, kMost>(s, b, at, s_beams, P.K);
  else if (s.unit == 4) move_column<uint32_t, kMost>(s, b, at, s_beams, P.K);
  else if (s.unit == 2) move_column<uint16_t, kMost>(s, b, at, s_beams, P.K);
  else move_column<uint8_t, kMost>(s, b, at, s_beams, P.K);
}

}  // namespace

extern "C" {

size_t specv_beam_workspace_bytes(int B, int W, int K, int V) {
  if (check_beams(B, W, K) != SPECV_OK || V < 1 || V > 1 << kVocabBits) return 0;
  return Plan(B, W, K, V).total;
}

specv_status spec_select_beams(const void* logits, int64_t batch_stride, int64_t row_stride,
                               specv_dtype dtype, int B, int W, int V, int K, const float* scores,
                               const int32_t* ended, int end_token, float* out_scores,
                               int32_t* tokens, int32_t* beams, int32_t* status, void* workspace,
                               size_t workspace_bytes, specv_stream_t stream) {
  const specv_status s = check_beams(B, W, K);
  if (s != SPECV_OK) return s;
  if (dtype != SPECV_F32 && dtype != SPECV_BF16) return SPECV_ERR_INVALID_ARG;
  if (!logits || !scores || !out_scores || !tokens || !beams || !status || !workspace || V < 1 ||
      batch_stride < 0 || row_stride < 0)
    return SPECV_ERR_INVALID_ARG;
  if (!aligned_to(logits, dtype == SPECV_F32 ? 4 : 2) || !aligned_to(scores, 4) ||
      !aligned_to(ended, 4) || !aligned_to(out_scores, 4) || !aligned_to(tokens, 4) ||
      !aligned_to(beams, 4) || !aligned_to(status, 4) || !aligned_to(workspace, 256))
    return SPECV_ERR_INVALID_ARG;
  if (V > specv_max_vocab(dtype)) return SPECV_ERR_UNSUPPORTED;
  const Plan plan(B, W, K, V);
  if (workspace_bytes < plan.total) return SPECV_ERR_WORKSPACE;
  char* base = static_cast<char*>(workspace);
  const Params P{logits,
                 batch_stride,
                 row_stride,
                 scores,
                 ended,
                 reinterpret_cast<Part*>(base),
                 reinterpret_cast<uint64_t*>(base + plan.keys),
                 out_scores,
                 tokens,
                 beams,
                 status,
                 W,
                 V,
                 K,
                 plan.splits,
                 plan.tiles,
                 end_token};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const unsigned blocks = static_cast<unsigned>(B) * W * plan.splits;
  if (dtype == SPECV_F32) select_rows_kernel<SPECV_F32><<<blocks, kThreads, 0, st>>>(P);
  else select_rows_kernel<SPECV_BF16><<<blocks, kThreads, 0, st>>>(P);
  if (launched() != SPECV_OK) return SPECV_ERR_CUDA;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(B);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, select_kernel, P) != cudaSuccess) {
    cudaGetLastError();
    return SPECV_ERR_CUDA;
  }
  return SPECV_OK;
}

specv_status spec_reorder_beams(const int32_t* beams, int B, int W, int K, const specv_state* states,
                                int num_states, int32_t* status, specv_stream_t stream) {
  const specv_status s = check_beams(B, W, K);
  if (s != SPECV_OK) return s;
  if (!beams || !states || !status || num_states < 1 || !aligned_to(beams, 4) || !aligned_to(status, 4))
    return SPECV_ERR_INVALID_ARG;
  if (num_states > SPECV_MAX_STATES) return SPECV_ERR_UNSUPPORTED;
  MoveParams P;
  P.beams = beams;
  P.status = status;
  P.W = W;
  P.K = K;
  P.states = num_states;
  const int most = K <= 16 ? 16 : K <= 32 ? 8 : 4;  // bytes of a column: K of them in registers
  int64_t tiles = 0;
  for (int i = 0; i < num_states; i++) {
    const specv_state& x = states[i];
    if (!x.in || !x.out || x.bytes < 1 || x.in_batch_stride < 0 || x.in_beam_stride < 0 ||
        x.out_batch_stride < 0 || x.out_beam_stride < 0 || (K > 1 && x.out_beam_stride < x.bytes) ||
        (x.in == x.out && (x.in_batch_stride != x.out_batch_stride ||
                           x.in_beam_stride != x.out_beam_stride)))
      return SPECV_ERR_INVALID_ARG;
    const uint64_t bits = reinterpret_cast<uintptr_t>(x.in) | reinterpret_cast<uintptr_t>(x.out) |
                          x.in_batch_stride | x.in_beam_stride | x.out_batch_stride |
                          x.out_beam_stride | x.bytes | most;
    const int unit = static_cast<int>(bits & (~bits + 1));
    P.state[i] = Moved{static_cast<const char*>(x.in), static_cast<char*>(x.out), x.in_batch_stride,
                       x.in_beam_stride, x.out_batch_stride, x.out_beam_stride, x.bytes,
                       unit, static_cast<int>(tiles)};
    tiles += (x.bytes / unit + kMoveThreads - 1) / kMoveThreads;
    if (tiles > INT_MAX) return SPECV_ERR_UNSUPPORTED;
  }
  // requests along two axes of the grid, of at most 65,535 blocks each
  const dim3 grid(static_cast<unsigned>(tiles), B < 32768 ? B : 32768, (B + 32767) / 32768);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (K <= 8) reorder_kernel<8><<<grid, kMoveThreads, 0, st>>>(P);
  else if (K <= 16) reorder_kernel<16><<<grid, kMoveThreads, 0, st>>>(P);
  else if (K <= 32) reorder_kernel<32><<<grid, kMoveThreads, 0, st>>>(P);
  else reorder_kernel<64><<<grid, kMoveThreads, 0, st>>>(P);
  return launched();
}

}  // extern "C"
