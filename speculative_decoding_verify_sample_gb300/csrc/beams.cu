// The drafting of a tree, or a beam search's step: the best of all beams' next
// tokens, and their states moved along.
//
//   score(w, v) = scores[w] + z[w,v] - log sum_u exp z[w,u],
//
// the K best of W V.  Within a row the order is that of z, so a block that has a part of a
// row keeps that part's K best entries and its sum of exponentials; a request's block then
// has the rows' sums, turns the parts' entries into scores and takes the K best of them.
// Each logit is read once, and only the few that may be among the best leave the
// registers.
//
// Measured: 64 requests of 8 beams over 128,256 32-bit entries, a fifth of them ended, 59 to 60
// us (210 MB, 3.5 TB/s), none ended 85 (263 MB): more rows than blocks fit at a time, 456, so the
// last 56 run by themselves (57 requests, 456 rows: 60).  Rows that do not begin at 16 bytes, as those of 128,257
// entries, 142 and 170.  One request of 8 over 16-bit entries 19 to 20; a single row of 1,024
// entries 12.4, two kernels' latencies.  32 requests of 16 beams, K = 16, 16 bits: 89;
// 8 of 64 over 50,000, K = 64: 177, nearly all of it the search.  What bounds the rows is not separated: in
// an earlier form of 98 us the batch took 59 without the search for the best and 51 without the
// exponentials as well.  The reordering of 64 requests of 8 beams, 46 MB read and written, 10.5 us, of one 4.

#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "cache.cuh"

using namespace specv_cache_ops;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kVecs = 4;  // vectors of 16 bytes that a lane has of a row at a time
constexpr int kMaxBeams = SPECV_MAX_BEAMS;
constexpr int kBuffer = 128;  // entries of a warp that may be among the best, until they are sorted in
constexpr int kFound = 1024;  // and of a request
constexpr int kKept = 8192;   // candidates that a request's block keeps in shared memory, at most
// Shared memory of a request's block where there are no more of them than SMs: an SM has one.  With only what
// it needs, how many an SM gets hangs on a few hundred bytes (why more are slower was not looked
// into): 32 requests of 16 beams, K = 16, 16 bits took 93 or 116 us for 3 or 4 KB more, and 89 so; 64 of 8,
// 32 bits, a fifth of them ended, 66 and 59; 16 of 16, K = 32, 98 and 63.  More requests than SMs:
// 200 of 2 beams 31 and 35, 1,000 of 4 151 and 176.
constexpr int kAlone = 100 * 1024;
constexpr int kVocabBits = 20;  // of a vocabulary entry's number
constexpr int kMaxSplits = 32;  // parts of a row: a request's block reads what they leave
constexpr int kBlocks = 3;     // of an SM, where rows are long enough

template <int DT> struct Elt;
template <> struct Elt<SPECV_F32> {
  using T = float;
  static constexpr int kVec = 4;
  static constexpr uint32_t kNone = 0xff800000u;  // -inf
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
  static constexpr uint32_t kNone = 0xff80ff80u;
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
  int kept;  // candidates that a request's block keeps in shared memory
  int W, V, K, splits, steps, end_token;  // parts of a row, steps of each of a part's warps
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

// The vector of a row's entries from `at` on, -inf behind the last, where it is not one of 16
// aligned bytes: two such are shifted together where both lie within the row.  (By itself, for
// its code is seldom needed and long.)
template <int DT>
__device__ __noinline__ uint4 load_odd(const typename Elt<DT>::T* row, int at, int V, int shift) {
  using E = Elt<DT>;
  constexpr int kVec = E::kVec, kSize = 16 / kVec;
  uint4 v = make_uint4(E::kNone, E::kNone, E::kNone, E::kNone);
  if (at >= V) return v;
  if (at * kSize >= shift && (at + 2 * kVec) * static_cast<int64_t>(kSize) - shift <= V * static_cast<int64_t>(kSize)) {
    const uint4* from = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(row + at) - shift);
    const uint4 a = __ldg(from), b = __ldg(from + 1);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t x[5];
    const int words = shift / 4;
#pragma unroll
    for (int i = 0; i < 5; i++)
      x[i] = words == 0 ? w[i] : words == 1 ? w[i + 1] : words == 2 ? w[i + 2] : w[i + 3];
#pragma unroll
    for (int i = 0; i < 4; i++) (&v.x)[i] = shift % 4 ? __funnelshift_r(x[i], x[i + 1], 16) : x[i];
  } else {
#pragma unroll
    for (int i = 0; i < kVec; i++)
      if (at + i < V) reinterpret_cast<typename E::T*>(&v)[i] = row[at + i];
  }
  return v;
}

// Adds how many of n keys are larger, two at a time (of an odd number one more is there, 0).
__device__ __forceinline__ void rank_among(const uint64_t* keys, int n, uint64_t key, int& rank) {
#pragma unroll 4
  for (int k = 0; k < n; k += 2) {
    const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(keys + k);
    rank += (two.x > key) + (two.y > key);
  }
}

// The K-th largest of a warp's 32 numbers (a bitonic sort).
__device__ __forceinline__ float kth_of_warp(float x, int K, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k *= 2)
#pragma unroll
    for (int j = k / 2; j > 0; j /= 2) {
      const float y = __shfl_xor_sync(kFullMask, x, j);
      x = ((lane & j) == 0) == ((lane & k) == 0) ? fmaxf(x, y) : fminf(x, y);
    }
  return __shfl_sync(kFullMask, x, K - 1);
}

// A number that K of a warp's 128, or a few more, are not below (-inf where fewer are finite).
__device__ __forceinline__ float about_kth_of_warp(const float (&x)[4], int K) {
  uint32_t key[4], low = 0, high = 0;
#pragma unroll
  for (int j = 0; j < 4; j++) {
    key[j] = x[j] > -INFINITY ? static_cast<uint32_t>(key_of(x[j], 0) >> 32) : 0;
    high = max(high, key[j]);
  }
  high = __reduce_max_sync(kFullMask, high);
  // low: K or more are not below; above high there are fewer
#pragma unroll 1
  while (low < high) {
    const uint32_t middle = low + (high - low + 1) / 2;
    int n = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) n += __popc(__ballot_sync(kFullMask, key[j] >= middle));
    if (n >= K) low = middle;
    else high = middle - 1;
    if (n >= K && n <= K + K / 4) break;
  }
  return low ? value_of(static_cast<uint64_t>(low) << 32) : -INFINITY;
}

// A block's part of one row.  Its warps go through it in steps, in turn, the next step's
// loads under way, and tell one another what no entry of the row's best can be below.
template <int DT>
__global__ void __launch_bounds__(kThreads, 3) select_rows_kernel(const Params P) {
  using E = Elt<DT>;
  constexpr int kVec = E::kVec, kMine = kVecs * kVec, kStep = 32 * kMine;
  __shared__ __align__(16) uint64_t s_best[kWarps][2][kMaxBeams + 2];
  __shared__ __align__(16) uint64_t s_found[kWarps][kBuffer + 2];
  __shared__ float s_max[kWarps];
  __shared__ double s_sum[kWarps];
  __shared__ __align__(16) uint64_t s_all[kWarps * kMaxBeams + 2];
  __shared__ uint32_t s_least;  // (as the upper half of a key)
  __shared__ float s_share[kWarps];  // a warp's best but K / kWarps
  __shared__ int s_count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  const int64_t row = blockIdx.x / P.splits;
  const int split = blockIdx.x - static_cast<int>(row) * P.splits, K = P.K;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // A beam that has ended or is not in play has no row.
  if (P.scores[row] == -INFINITY || (P.ended && P.ended[row])) return;
  const auto* from = static_cast<const typename E::T*>(P.logits) + row / P.W * P.batch_stride +
                     row % P.W * P.row_stride;
  const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(from) & 15);
  uint64_t* const found = s_found[warp];
  if (tid == 0) {
    s_least = 0;
    s_count = 0;
  }
  if (tid < kWarps) s_share[tid] = -INFINITY;
  const int share = (K + kWarps - 1) / kWarps;
  __syncthreads();

  // Of this lane's entries; their sum is l + rest, what l's roundings leave out kept beside it, so that a
  // row's sum has twice 32 bits (64 requests of 8 beams of 128,256 entries: 67 us, one number of 64 bits 68,
  // l alone 65, but 2^-19 off for rows of 500,000 equal steps)
  float m = -INFINITY, l = 0.0f, rest = 0.0f;
  int have = 0, now = 0;  // entries of s_best[now]
  int waiting = 0;        // entries of found
  // What is below `least`, or equal and not in front of `least_at`, is not among the K best.
  float least = -INFINITY;
  int least_at = -1;
  auto tell = [&]() {
    if (lane == 0 && least > -INFINITY) atomicMax(&s_least, static_cast<uint32_t>(key_of(least, 0) >> 32));
  };
  // Sorts the found entries in: each goes to the place that its rank is.
  auto merge = [&]() {
    if (lane == 0) {  // (pairs are compared: behind the last a key that is below all)
      found[waiting] = 0;
      s_best[warp][now][have] = 0;
    }
    __syncwarp();
    const int all = have + waiting;
    const uint64_t* best = s_best[warp][now];
    uint64_t* to = s_best[warp][now ^ 1];
    for (int i = lane; i < all; i += 32) {
      const uint64_t key = i < have ? best[i] : found[i - have];
      int rank = 0;
      rank_among(best, have, key, rank);
      rank_among(found, waiting, key, rank);
      if (rank < K) to[rank] = key;
    }
    __syncwarp();
    have = min(K, all);
    now ^= 1;
    waiting = 0;
    if (lane == 0 && have >= share) static_cast<volatile float*>(s_share)[warp] = value_of(to[share - 1]);
    if (have == K) {
      const uint64_t last = to[K - 1];
      if (value_of(last) >= least) {
        least = value_of(last);
        least_at = place_of(last);
        tell();
      }
    }
  };

  const int begin = split * P.steps * kWarps * kStep;
  const int whole = shift ? 0 : P.V;  // entries in aligned vectors
  uint4 next[2][kVecs];  // of this step and the one behind it
  auto first_of = [&](int step) { return begin + (step * kWarps + warp) * kStep; };
  auto fetch = [&](int step, uint4 (&to)[kVecs]) {
#pragma unroll
    for (int j = 0; j < kVecs; j++) {
      const int e = first_of(step) + (j * 32 + lane) * kVec;
      if (step < P.steps && e + kVec <= whole) to[j] = __ldg(reinterpret_cast<const uint4*>(from + e));
      else to[j] = step < P.steps && e < P.V ? load_odd<DT>(from, e, P.V, shift)
                                             : make_uint4(E::kNone, E::kNone, E::kNone, E::kNone);
    }
  };
  fetch(0, next[0]);
  fetch(1, next[1]);
#pragma unroll 1
  for (int step = 0; step < P.steps; step++) {
    const int first = first_of(step);
    if (first >= P.V) break;
    float z[kMine], tops[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; j++) {
      E::unpack(next[0][j], z + j * kVec);
      next[0][j] = next[1][j];
    }
    fetch(step + 2, next[1]);
#pragma unroll
    for (int j = 0; j < kVecs; j++) {
      tops[j] = z[j * kVec];
#pragma unroll
      for (int e = 1; e < kVec; e++) tops[j] = fmaxf(tops[j], z[j * kVec + e]);
    }
    const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    // (a NaN or +inf makes the sum a NaN, which the request's block sees)
    const float higher = fmaxf(m, top), from_max = higher == -INFINITY ? 0.0f : higher;
    float sums[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < kMine; j++) sums[j % 4] += exp_of(z[j] - from_max);
    const float by = m == higher ? 1.0f : exp_of(m - higher), more = (sums[0] + sums[1]) + (sums[2] + sums[3]);
    l *= by;
    const float next_l = l + more, added = next_l - l;
    rest = fmaf(rest, by, (l - (next_l - added)) + (more - added));
    l = next_l;
    m = higher;

    if (step == 0) {
      // The K-th largest of the lanes' maxima, or of all vectors': as many entries are not below it.
      const float kth = K <= 8 ? kth_of_warp(top, K, lane) : about_kth_of_warp(tops, K);
      least = kth;
      least_at = kth > -INFINITY ? INT_MAX : -1;
      tell();
    }
    // Nothing below another warp's K-th best is among the row's, nor below the least of what all
    // warps have K / kWarps entries of.
    const uint32_t told = *static_cast<volatile uint32_t*>(&s_least);
    float others = static_cast<volatile float*>(s_share)[lane % kWarps];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o /= 2) others = fminf(others, __shfl_xor_sync(kFullMask, others, o));
    if (told) others = fmaxf(others, value_of(static_cast<uint64_t>(told) << 32));
    if (others > least) {
      least = others;
      least_at = INT_MAX;
    }
    if (!__any_sync(kFullMask, top >= least && top > -INFINITY)) continue;
    // The entries not below it, each lane its own one after the other, read once more.  (Short
    // code: a block that goes through this once or twice spends its time on fetching it.)
    uint32_t mask = 0;
#pragma unroll
    for (int e = 0; e < kMine; e++) mask |= z[e] >= least ? 1u << e : 0u;
#pragma unroll 1
    while (__any_sync(kFullMask, mask != 0)) {
      const int e = mask ? __ffs(mask) - 1 : 0;
      const int place = first + (e / kVec * 32 + lane) * kVec + e % kVec;
      const float x = mask && place < P.V ? E::one(from[place]) : -INFINITY;
      mask &= mask - 1;
      unsigned good = __ballot_sync(kFullMask, x > least || (x == least && place < least_at));
      if (waiting + __popc(good) > kBuffer) {
        merge();
        good = __ballot_sync(kFullMask, x > least || (x == least && place < least_at));
      }
      if (good >> lane & 1) found[waiting + __popc(good & ((1u << lane) - 1))] = key_of(x, place);
      waiting += __popc(good);
    }
    if (waiting) merge();
  }
  // The part's maximum and sum, and the best of the warps' best.
  float all = m;
#pragma unroll
  for (int o = 16; o > 0; o /= 2) all = fmaxf(all, __shfl_xor_sync(kFullMask, all, o));
  double sum = static_cast<double>(l) + static_cast<double>(rest);
  if (m != all) sum *= static_cast<double>(exp_of(m - all));
#pragma unroll
  for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(kFullMask, sum, o);
  int at = 0;
  if (lane == 0) {
    s_max[warp] = all;
    s_sum[warp] = sum;
    at = atomicAdd(&s_count, have);
  }
  at = __shfl_sync(kFullMask, at, 0);
  for (int k = lane; k < have; k += 32) s_all[at + k] = s_best[warp][now][k];
  __syncthreads();
  const int64_t part = blockIdx.x;
  const int n = s_count;
  if (n % 2) {
    if (tid == 0) s_all[n] = 0;
    __syncthreads();
  }
  for (int i = tid; i < n; i += kThreads) {
    const uint64_t key = s_all[i];
    int rank = 0;
    rank_among(s_all, n, key, rank);
    if (rank < K) P.keys[part * K + rank] = key;
  }
  for (int k = n + tid; k < K; k += kThreads) P.keys[part * K + k] = 0;
  if (tid == 0) {
    float most = s_max[0];
    for (int w = 1; w < kWarps; w++) most = fmaxf(most, s_max[w]);
    double total = 0.0;
    for (int w = 0; w < kWarps; w++)
      total += s_max[w] == most ? s_sum[w] : s_sum[w] * static_cast<double>(exp_of(s_max[w] - most));
    P.parts[part] = Part{most, 0.0f, total};
  }
}

// A candidate: its score as a whole number of the same order, and what decides between equal ones,
// the larger first: the lower beam, the larger logit (of one beam's entries the score falls
// with it, also where a sum far from 0, a score of -1e30, leaves no difference in 64 bits, and a
// part's list is in that order), the lower token.
struct Candidate {
  uint64_t score;  // kNothing: none
  uint64_t tie;
};
constexpr uint32_t kLastEntry = (1u << kVocabBits) - 1;
static_assert((kMaxBeams & (kMaxBeams - 1)) == 0 && kMaxBeams <= 1 << (32 - kVocabBits), "bits of a tie");
__device__ __forceinline__ uint64_t tie_of(int w, uint32_t logit, int token) {
  return static_cast<uint64_t>(kMaxBeams - 1 - w) << (32 + kVocabBits) |
         static_cast<uint64_t>(logit) << kVocabBits | (kLastEntry - static_cast<uint32_t>(token));
}
__device__ __forceinline__ int beam_of(uint64_t tie) {
  return kMaxBeams - 1 - static_cast<int>(tie >> (32 + kVocabBits));
}
__device__ __forceinline__ int token_of(uint64_t tie) {
  return static_cast<int>(kLastEntry - (static_cast<uint32_t>(tie) & kLastEntry));
}
constexpr uint64_t kNothing = 0x000fffffffffffffull;  // of -inf
__device__ __forceinline__ uint64_t ordered(double x) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));  // (-0 is 0)
  return u >> 63 ? ~u : u | 1ull << 63;
}
__device__ __forceinline__ double score_of(uint64_t u) {
  return __longlong_as_double(static_cast<long long>(u >> 63 ? u & ~(1ull << 63) : ~u));
}
__device__ __forceinline__ bool better(const Candidate& a, const Candidate& b) {
  return a.score > b.score || (a.score == b.score && a.tie > b.tie);
}
__device__ __forceinline__ uint64_t larger(uint64_t a, uint64_t b) { return a > b ? a : b; }

// A request's block: the rows' sums, then the K best of the parts' entries.
__global__ void __launch_bounds__(kThreads) select_kernel(const Params P) {
  __shared__ double s_off[kMaxBeams];  // score - log sum of a row; an ended beam's score
  __shared__ float s_max[kMaxBeams];   // and what that sum's exponentials were taken from
  __shared__ uint8_t s_kind[kMaxBeams];  // 0: no candidate, 1: a row, 2: ended
  __shared__ Candidate s_found[kFound];
  extern __shared__ __align__(16) uint64_t s_score[];  // [kept], and behind them what decides ties
  uint64_t* const s_tie = s_score + P.kept;
  __shared__ uint64_t s_top[kMaxBeams];
  __shared__ Candidate s_warp[kWarps];
  __shared__ int s_count, s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  const int64_t b = blockIdx.x;
  const int W = P.W, K = P.K;
  if (tid == 0) s_count = s_bad = 0;
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int w = warp; w < W; w += kWarps) {
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
        sum += part.max == m ? part.sum : part.sum * static_cast<double>(part.max == -INFINITY ? 0.0f : exp_of(part.max - m));
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
  const bool bad = s_bad != 0;
  const int lists = W * P.splits, all = bad ? 0 : lists * K;
  // Entry number e; worse than any where there is none.  The lists' first entries come first, those
  // of all rows beside one another, so that every group of threads below has good ones.
  const Candidate none{kNothing, 0};
  auto entry = [&](int e) {
    const int k = e / lists, list = e - k * lists, split = list / W, w = list - split * W, kind = s_kind[w];
    Candidate c = none;
    if (kind == 1) {
      const uint64_t key = P.keys[((b * W + w) * P.splits + split) * K + k];
      if (key) {
        c.score = ordered(s_off[w] + (static_cast<double>(value_of(key)) - static_cast<double>(s_max[w])));
        c.tie = tie_of(w, static_cast<uint32_t>(key >> 32), place_of(key));
      }
    } else if (kind == 2 && !k && !split) {
      c.score = ordered(s_off[w]);
      c.tie = tie_of(w, 0, 0);
    }
    return c;
  };
  // The least of K or more groups' best: nothing below it is among the K best.
  uint64_t mine = kNothing;
#pragma unroll 1
  for (int e = tid; e < all; e += kThreads) {
    const Candidate c = entry(e);
    if (e < P.kept) {
      s_score[e] = c.score;
      s_tie[e] = c.tie;
    }
    mine = larger(mine, c.score);
  }
  // (a thread's own, no other's)
  auto again = [&](int e) { return e < P.kept ? Candidate{s_score[e], s_tie[e]} : entry(e); };
  const int groups = K <= 8 ? 8 : K <= 16 ? 16 : K <= 32 ? 32 : 64, width = kThreads / groups;
  for (int o = width / 2; o > 0; o /= 2) mine = larger(mine, __shfl_xor_sync(kFullMask, mine, o));
  if (tid % width == 0) s_top[tid / width] = mine;
  __syncthreads();
  uint64_t least = s_top[0];
#pragma unroll 1
  for (int g = 1; g < groups; g++) least = s_top[g] < least ? s_top[g] : least;
  auto collect = [&]() {
#pragma unroll 1
    for (int e = tid; e < all; e += kThreads) {
      const Candidate c = again(e);
      if (c.score <= kNothing || c.score < least) continue;
      const int at = atomicAdd(&s_count, 1);
      if (at < kFound) s_found[at] = c;
    }
  };
  collect();
  __syncthreads();
  int found = s_count;
  const int enough = min(kFound, 4 * K + 64);
  if (found > enough) {
    // Too many: halve what lies between that bound and the best until the bound leaves few enough.
    uint64_t low = least, high = s_top[0];  // low leaves K or more, high fewer than that or too few
    for (int g = 1; g < groups; g++) high = larger(high, s_top[g]);
    while (found > enough && high - low > 1) {
      const uint64_t middle = low + (high - low) / 2;
      int n = 0;
#pragma unroll 1
      for (int e = tid; e < all; e += kThreads) n += again(e).score >= middle;
      __syncthreads();
      if (tid == 0) s_count = 0;
      __syncthreads();
      n = __reduce_add_sync(kFullMask, n);
      if (lane == 0 && n) atomicAdd(&s_count, n);
      __syncthreads();
      if (s_count >= K) {
        low = middle;
        found = s_count;
      } else {
        high = middle;
      }
    }
    least = low;
    __syncthreads();
    if (tid == 0) s_count = 0;
    __syncthreads();
    if (found <= kFound) collect();
    __syncthreads();
  }
  auto put = [&](int k, const Candidate& c) {
    // (a score below the lowest 32-bit number is out of play behind this call, as one of -inf)
    const float score = c.score > kNothing ? static_cast<float>(score_of(c.score)) : -INFINITY;
    const bool real = score > -INFINITY;
    const int w = real ? beam_of(c.tie) : 0;
    P.out_scores[b * K + k] = score;
    P.beams[b * K + k] = real ? w : -1;
    P.tokens[b * K + k] = !real ? -1 : s_kind[w] == 2 ? P.end_token : token_of(c.tie);
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
    // Still too many (scores all alike): one after the other, each the best of those behind the last.
    Candidate last{~0ull, 0};
    for (int k = 0; k < K; k++) {
      Candidate c = none;
      for (int e = tid; e < all; e += kThreads) {
        const Candidate d = again(e);
        if (better(last, d) && better(d, c)) c = d;
      }
#pragma unroll
      for (int o = 16; o > 0; o /= 2) {
        const Candidate d{__shfl_xor_sync(kFullMask, c.score, o), __shfl_xor_sync(kFullMask, c.tie, o)};
        if (better(d, c)) c = d;
      }
      if (lane == 0) s_warp[warp] = c;
      __syncthreads();
      c = s_warp[0];
      for (int i = 1; i < kWarps; i++)
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
  int steps, splits;  // of a part's warps; parts of a row
  size_t keys, total;

  Plan(int B, int W, int K, int V, int step) {
    const int all = (V + step * kWarps - 1) / (step * kWarps);  // steps of eight warps
    const int64_t rows = static_cast<int64_t>(B) * W, wanted = kBlocks * kSms;
    int64_t parts = (wanted + rows - 1) / rows;
    if (parts > kMaxSplits) parts = kMaxSplits;
    if (parts > all) parts = all;
    steps = static_cast<int>((all + parts - 1) / parts);
    splits = (all + steps - 1) / steps;
    keys = align256(rows * splits * sizeof(Part));
    total = keys + align256(rows * splits * K * sizeof(uint64_t));
  }

  // Enough for every call of up to B, W, K and V: fewer rows have more parts each, at most kMaxSplits
  // and at most this many in all, for parts < wanted / rows + 1.
  static size_t most(int B, int W, int K, int V, int step) {
    const int64_t rows = static_cast<int64_t>(B) * W, all = (V + step * kWarps - 1) / (step * kWarps);
    const int64_t each = rows * (all < kMaxSplits ? all : kMaxSplits), dealt = rows + kBlocks * kSms - 1;
    const int64_t parts = each < dealt ? each : dealt;
    return align256(parts * sizeof(Part)) + align256(parts * K * sizeof(uint64_t));
  }
};
template <int DT> constexpr int kStepOf = 32 * kVecs * Elt<DT>::kVec;

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
  int B, W, K, states;
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
  if (b >= P.B) return;
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

// Where a state's beams lie: `bytes` bytes at + b batch + w beam, for b < B and w < beams.
struct Places {
  __int128 at, end, batch, beam, bytes;
  int B, beams;

  Places(const void* p, int64_t batch_stride, int64_t beam_stride, int64_t bytes, int B, int beams)
      : at(reinterpret_cast<uintptr_t>(p)), batch(B > 1 ? batch_stride : 0), beam(beam_stride), bytes(bytes), B(B),
        beams(beams) {
    end = at + (B - 1) * batch + (beams - 1) * beam + bytes;
  }
};

// Whether two states' places have a byte in common.  Exact for strides that are alike, as those of views
// of one tensor are; others are only known to if they begin together.
bool overlap(const Places& x, const Places& y) {
  if (x.at == y.at) return true;
  if (x.end <= y.at || y.end <= x.at) return false;
  const __int128 beam = x.beams > 1 ? x.beam : y.beam, most = x.B - 1;
  if ((y.beams > 1 && y.beam != beam) || x.batch != y.batch) return false;
  for (int w = 1 - x.beams; w < y.beams; w++) {  // y's beam less x's
    // y's place less x's is `off` and b batches more: the first that is not wholly below
    const __int128 off = y.at - x.at + w * beam;
    __int128 b = -most;
    if (x.batch > 0) {
      const __int128 past = -y.bytes - off;  // b batch is above it
      const __int128 first = past / x.batch - (past % x.batch < 0) + 1;
      if (b < first) b = first;
    }
    const __int128 from = off + b * x.batch;
    if (b <= most && from > -y.bytes && from < x.bytes) return true;
  }
  return false;
}

}  // namespace

extern "C" {

size_t specv_beam_workspace_bytes(int B, int W, int K, int V) {
  if (check_beams(B, W, K) != SPECV_OK || V < 1 || V > 1 << kVocabBits) return 0;
  return Plan::most(B, W, K, V, kStepOf<SPECV_F32>);  // (a 16-bit row has no more steps)
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
  const Plan plan(B, W, K, V, dtype == SPECV_F32 ? kStepOf<SPECV_F32> : kStepOf<SPECV_BF16>);
  if (workspace_bytes < plan.total) return SPECV_ERR_WORKSPACE;
  char* base = static_cast<char*>(workspace);
  const int all = W * K * plan.splits, kept = (all < kKept ? all : kKept) + 1 & ~1;
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
                 kept,
                 W,
                 V,
                 K,
                 plan.splits,
                 plan.steps,
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
  cfg.dynamicSmemBytes = kept * sizeof(Candidate);
  if (B <= kSms && cfg.dynamicSmemBytes < kAlone) cfg.dynamicSmemBytes = kAlone;
  if (cfg.dynamicSmemBytes > 16384 &&
      cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kKept * sizeof(Candidate))) != cudaSuccess) {
    cudaGetLastError();
    return SPECV_ERR_CUDA;
  }
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
  P.B = B;
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
  // What one state's blocks write must not be what another's, or they themselves, still have to read.
  for (int i = 0; i < num_states; i++) {
    const specv_state& x = states[i];
    const Places to(x.out, x.out_batch_stride, x.out_beam_stride, x.bytes, B, K);
    for (int j = 0; j < num_states; j++) {
      const specv_state& y = states[j];
      if ((j < i && overlap(to, Places(y.out, y.out_batch_stride, y.out_beam_stride, y.bytes, B, K))) ||
          ((j != i || x.in != x.out) &&
           overlap(to, Places(y.in, y.in_batch_stride, y.in_beam_stride, y.bytes, B, W))))
        return SPECV_ERR_INVALID_ARG;
    }
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
