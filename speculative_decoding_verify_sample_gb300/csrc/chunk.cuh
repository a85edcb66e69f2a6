// Attention of chunks of new tokens over the paged cache.
//
// For one key head h of one request the query rows are the (token, query head)
// pairs of its group, G to a token.  256 of them are an item, its work the
// 128-key tiles that one of its tokens sees:
//
//   S = Q K^T (tcgen05, operands in shared memory, S in TMEM),
//   Y = cap tanh(scale S / cap) - slope |distance|, in units of log 2,
//   P = exp2(Y - m), m the running row maximum,
//   O = O + P V (tcgen05, P from TMEM where S was, V in shared memory),
//
// O rescaled only when the maximum has risen by more than 2^8: m is whatever both O
// and the sum l were taken with.
//
// An item's tiles are those below its prefix and then those from its window on;
// what lies between is not read.  Items' tiles are cut into even runs, one for
// every CTA (one to an SM), whatever the lengths are.  An item whose tiles one run
// has whole is written out; pieces leave (m, l, O) in the workspace for
// join_kernel.
//
// Two streams share an SM, each with its S and O in TMEM and its four softmax
// warps: an item of more than 128 rows is a pair of row tiles on the same keys, one of
// fewer shares its half tiles out to both and is joined at the end.  A stream's scores are
// taken half a tile (64 keys) at a time into two places in turn, so that the tensor cores
// can have the next half's scores done when the softmax has done with one.  The price:
// products of 64 keys read the queries from shared memory as often as those of 128, and two
// streams' scores and sums of a tile take the tensor cores 2,478 cycles in place of 2,050 (the
// MMAs alone, timed); tensor memory has no room for two whole tiles of scores and the sums.
// Besides the softmax there are four warps that copy, a warp to each stream's scores and one to
// its sums, one that lists the run's work, one that checks the requests' data and two
// that clean values.
//
// Measured (D = 128 and 32 + 8 heads but where said), calls back to back:
// 4,093 tokens behind 28,673 slots 1,423 to 1,452 us (1,430 TFLOP/s);
// six prompts of 517 to 4,093 tokens 327 us (1,020 TFLOP/s).  With clocks read in the
// kernel a softmax warp of this case has 22 halves to an item, each 150 cycles before its wait, 490
// in it and 950 at work, and 8,000 cycles at an item's ends, 5,200 of them writing (without the
// writes 315 us);
// 48 requests of 1 to 257 tokens and a window, f16, 185 us;
// single tokens: 48 over 27,000 slots each 780 us (6.8 TB/s), 64 over 4,001 174, 16 over 2,000 to 5,750 62, one
// over 32,001 42, over 4,001 in a table of 16,384 20 (in one of 4,032 it is the small kernel's, 12.4);
// capped scores, 16 + 8 heads, 297 us for 202 GFLOP: the polynomial's
// products come on top of each score's exponential;
// a bias by distance, 16 + 16 heads of 64, 138 to 140 us for 49 GFLOP (116 without the bias).
// The second kernel takes 18 to 41 us where items are many (under a profiler): its 197 registers to a thread
// leave an SM one block.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "cache.cuh"
#include "tensor.cuh"

namespace specv_chunk {

using namespace specv_cache_ops;
using namespace specv_tensor;

constexpr int kKeys = 128;     // keys of a tile
constexpr int kHalf = 64;      // and of its halves, whose scores are taken one at a time
constexpr int kRows = 128;     // query rows of a stream
constexpr int kRowTile = 256;  // and of an item
static_assert(kKeys == kRows, "tiles of queries, keys and values are laid out alike");
constexpr int kMaxCtas = kSms;
constexpr int kMaxRequests = SPECV_MAX_CHUNK_REQUESTS;
constexpr int kLoadWarps = 4;
constexpr int kLoadWarp = 8;    // the first of them; the last makes the tensor copies
constexpr int kScoreWarp = 12;  // two, a stream each: issue S = Q K^T
constexpr int kSumWarp = 14;    // two: issue O += P V
constexpr int kListWarp = 16;
constexpr int kCheckWarp = 17;
constexpr int kCleanWarp = 18;  // two: look at values that not every row sees
constexpr int kThreads = 640;
constexpr int kItems = 4;  // items listed ahead
// Units of work: a pair's tile is two, a single row tile's one.  What an item takes besides its
// tiles, its end and the next one's first scores (a mixed batch with 6 and 3, 6 and 5, 6 and 8, 10
// and 8: 213, 199, 186, 187 us; first chunks with 4, 6, 8, 10, 14 for pairs: 360, 333, 326, 328,
// 340; a key head to each query head 154, 145, 136, 137, 136):
constexpr int kPairCost = 8, kSingleCost = 8;
// Registers a thread of each warpgroup: 2 * 144 + 72 + 2 * 56 <= 480 = 5 * 96, what
// the block is launched with.  The softmax keeps half a tile's scores of a row in them.
#define SPECV_CHUNK_REGS_SOFTMAX "144"
#define SPECV_CHUNK_REGS_LOAD "72"
#define SPECV_CHUNK_REGS_OTHER "56"
constexpr float kRise = 8.0f;  // log2 of how far a maximum may rise before O is rescaled

// Where a run begins in the middle of an item: the item's second piece.  And
// whether one of the run's waits gave up, so that it may have left items undone.
struct Cut {
  int32_t b, h, row_tile, rows, first;  // first: the request's first packed row
  int32_t pieces;  // of the item; 0: the run does not begin with an item's second piece
  int32_t gave_up;
  int32_t pad;
};

struct Workspace {
  Cut* cuts;      // [runs]
  float2* stats;  // [2 runs][part_rows] pieces' m and l: of an item that began before the
                  // run, then of one that goes on behind it
  float4* parts;  // [2 runs][dim / 4][part_rows] their O, four columns of a row together: the
                  // softmax's lanes have a row each, and adjacent rows make whole lines
};

struct Params {
  Cache cache;
  Rows q, out;  // packed: node_stride is a token's
  Workspace ws;
  const int32_t* cu_tokens;
  const int32_t* prefix_lens;
  const float* slopes;
  int32_t* status;
  int B, T, longest, q_heads, group;  // group: query heads to a key head
  int window;                         // INT_MAX: none
  int ctas;                           // and runs
  int part_rows;                      // rows of a piece in the workspace
  int box_rows;                       // rows that one tensor copy brings; 0: copies of 16 bytes
  float scale_log2;                   // scale log2 e
  float cap_log2, cap_unit;           // cap log2 e and scale / cap; 0: no cap
  float cap_small;                    // products up to here take the polynomial, ...
  float cap_poly[5];                  // in the square of the product over the cap, times that
};

// One request's place: its packed rows, its slots, the prefix that all its tokens see.
struct Request {
  int first, n, len, prefix;
  unsigned bad;
};

__device__ __forceinline__ Request request_of(const Params& P, int b) {
  Request r;
  r.first = P.cu_tokens[b];
  const int last = P.cu_tokens[b + 1];
  r.len = P.cache.lens[b];
  const int prefix = P.prefix_lens ? P.prefix_lens[b] : 0;
  const int64_t slots = static_cast<int64_t>(P.cache.max_pages) * P.cache.page_size;
  r.bad = 0;
  const int64_t n = static_cast<int64_t>(last) - r.first;
  if (r.first < 0 || n < 0 || last > P.T || n > P.longest) r.bad |= SPECV_DEV_BAD_DRAFT_LEN;
  // (rows of a request with too many tokens are its own all the same)
  r.n = r.first < 0 || n < 0 || last > P.T ? 0 : static_cast<int>(n);
  if (r.len < 0 || r.len + static_cast<int64_t>(r.n) > slots ||
      r.len + static_cast<int64_t>(r.n) > INT_MAX - 1024 || prefix < 0)
    r.bad |= SPECV_DEV_BAD_CACHE;
  r.prefix = r.bad ? 0 : min(prefix, r.len + r.n);
  return r;
}

// The first slot in the window of the token at pos.
__host__ __device__ __forceinline__ int lowest(const Params& P, int pos) {
  return P.window > pos ? 0 : pos - P.window + 1;
}

// The 128-key tiles of an item: numbers 0 .. tiles-1, tile i being keys from
// 128 i on, or 128 (i + skip) from number `gap` on.
struct Span {
  int rows, pos0, pos1, tiles, gap, skip;
};

__host__ __device__ __forceinline__ Span span_of(const Params& P, const Request& r, int row_tile) {
  Span s;
  const int all = r.n * P.group, at = row_tile * kRowTile;
  s.rows = min(kRowTile, all - at);
  s.pos0 = r.len + at / P.group;
  s.pos1 = r.len + (at + s.rows - 1) / P.group;
  s.gap = (r.prefix + kKeys - 1) / kKeys;
  s.skip = max(0, lowest(P, s.pos0) / kKeys - s.gap);
  s.tiles = max(s.gap, s.pos1 / kKeys + 1) - s.skip;
  return s;
}

// An item's units of work: what it takes besides its tiles, and they.
__device__ __forceinline__ int cost_of(const Span& s) { return s.rows > kRows ? kPairCost : kSingleCost; }
__device__ __forceinline__ int units_of(const Span& s) {
  return cost_of(s) + s.tiles * (s.rows > kRows ? 2 : 1);
}

__device__ __forceinline__ int row_tiles_of(const Params& P, const Request& r) {
  return r.bad ? 0 : (r.n * P.group + kRowTile - 1) / kRowTile;
}

// One key head's units of request r, the whole warp together.
__device__ __forceinline__ int64_t head_units(const Params& P, const Request& r, int lane) {
  const int R = row_tiles_of(P, r);
  int64_t sum = 0;
  for (int k = lane; k < R; k += 32) sum += units_of(span_of(P, r, k));
#pragma unroll
  for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(kFullMask, sum, o);
  return sum;
}

// How the units are cut into runs: a tile is the run's in which its first unit lies.
// (At least as long as a pair's tile, so that every run between an item's first and
// last has tiles of it.)
struct Runs {
  int64_t total, each;

  __device__ __forceinline__ Runs(const Params& P, int64_t units)
      : total(units), each(max(static_cast<int64_t>(2), quotient(units + P.ctas - 1, P.ctas))) {}
  static __device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return (a | b) >> 32 ? a / b : static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  }
  // Where run `run` begins, and run - 1 ends.
  __device__ __forceinline__ int64_t start(int run) const { return min(total, run * each); }
  // The run that has unit u.
  __device__ __forceinline__ int of(int64_t u) const { return static_cast<int>(quotient(u, each)); }
};

// The n lowest bits.
__device__ __forceinline__ uint32_t bits_below(int n) {
  return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one)::"memory");
  return one;
}

__device__ __forceinline__ float rcp_of(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int DP> struct Shape {
  static constexpr int kTileBytes = kKeys * DP * 2;  // of keys or of values
  static constexpr int kQueryBytes = kRows * DP * 2;
  static constexpr int kStages = 5 * (128 / DP);
  // shared memory: two tiles of queries (a pair's, or this and the next item's), stages,
  // then the barriers and what the warps tell one another
  static constexpr int kStageAt = 2 * kQueryBytes;
  static constexpr int kTailAt = kStageAt + kStages * kTileBytes;
  static_assert(kStages * kTileBytes >= kMaxRequests * 8, "requests' units lie there at first");

  // The order of an item's tiles in the ring: keys a tile ahead of values, K0 K1 V0 K2 V1 ..
  // Kn Vn-1 Vn, as scores are taken half a tile or more ahead of the sums.
  static __device__ __forceinline__ uint32_t key_job(int i) { return i ? 2 * i - 1 : 0; }
  static __device__ __forceinline__ uint32_t value_job(int i, int tiles) {
    return i == tiles - 1 ? 2 * i + 1 : 2 * i + 2;
  }
};

// Keys that some rows of an item see and others do not: behind the first row's
// own (up to 255), and below the last row's window (as many).  A bit each.
constexpr int kEdge = 8;

// Tiles number t0 .. t1-1 of an item that one run has.  They are taken from the last
// to the first, each from its upper half: a bias by distance is least there, so
// maxima are found early.
struct Item {
  int32_t b, h, row_tile, t0, t1, gap, skip, rows;  // t0 < 0: no more items
  int32_t first, n, len, prefix;
  int32_t pos0, pos1, low0, low1;  // positions and lowest slots of its first and last row
  int32_t pieces;  // runs that have tiles of it
  int32_t begins;  // this is its first piece
  int32_t bad;     // written by the checking warp
  int32_t any_odd;          // some edge keys' values were not finite:
  uint32_t odd[2 * kEdge];  // which
};

// An item's keys as a thread has them in registers.
struct Keys {
  int tiles, last, gap, skip, prefix, pos0, pos1, low0, low1;

  __host__ __device__ __forceinline__ explicit Keys(const Item& w)
      : tiles(w.t1 - w.t0), last(w.t1 - 1), gap(w.gap), skip(w.skip), prefix(w.prefix), pos0(w.pos0),
        pos1(w.pos1), low0(w.low0), low1(w.low1) {}
  // Makes them known to be the same in every lane.
  __device__ __forceinline__ void same() {
    for (int* x : {&tiles, &last, &gap, &skip, &prefix, &pos0, &pos1, &low0, &low1})
      *x = __shfl_sync(kFullMask, *x, 0);
  }
  // The first key of the i-th tile taken.
  __host__ __device__ __forceinline__ int first(int i) const {
    const int t = last - i;
    return (t < gap ? t : t + skip) * kKeys;
  }
  // Whether not every row sees all of these keys.
  __device__ __forceinline__ bool mixed(int key0, int n) const {
    return !((key0 + n <= prefix) | ((key0 >= low1) & (key0 + n - 1 <= pos0)));
  }
};

// The halves of its tiles in which some row sees a key, in the order in which they are taken:
// `total` of them, the first `turn` down from key `top`, the others, a prefix's, from `top2`.
struct Halves {
  int total, turn, top, top2;

  __host__ __device__ __forceinline__ Halves(const Keys& k, int t0) {
    const int t1 = t0 + k.tiles;
    const int own = (k.prefix + kHalf - 1) / kHalf;  // of the prefix
    int low = k.low0 / kHalf, high = k.pos1 / kHalf;
    const bool joined = own > 0 && own >= low;  // the window's follow on the prefix's
    if (joined) {
      low = 0;
      high = max(high, own - 1);
    }
    high = min(high, 2 * (t1 + k.skip) - 1);
    turn = max(0, high - max(low, 2 * (t0 + k.skip)) + 1);
    top = high * kHalf;
    const int last = min(own, 2 * t1) - 1;
    total = turn + (joined ? 0 : max(0, last - 2 * t0 + 1));
    top2 = last * kHalf;
  }
  __host__ __device__ __forceinline__ int key(int i) const {
    return i < turn ? top - i * kHalf : top2 - (i - turn) * kHalf;
  }
  // How many of them stream st takes: all of a pair's, of one row tile's every other one.
  __host__ __device__ __forceinline__ int taken(bool pair, int st) const {
    return pair ? total : (total + 1 - st) / 2;
  }
  // Whether stream st's sums are in the rows that stream `of_rows` writes at the item's end.  Made of
  // what all lanes know alike, for tensor memory is read by whole warps; and of an item that is
  // flagged, or behind a wait that gave up, nothing is read.
  __host__ __device__ __forceinline__ bool summed(bool pair, int of_rows, int st, bool bad) const {
    return !bad && (!pair || of_rows == st) && taken(pair, st) > 0;
  }
};

// A stream's scores lie in two halves of its part of TMEM in turn, so that the next ones
// are there when the softmax has done with one.
template <int kStages> struct Tail {
  uint64_t kv_full[kStages], kv_clean[kStages], kv_empty[kStages], q_full[2], q_empty[2];
  uint64_t s_full[2][2], p_full[2][2], o_full[2][2];  // by stream and half
  uint64_t item_full[kItems], item_checked[kItems], item_empty[kItems];
  uint64_t joined, parted;  // both streams at the end of an item that they share
  uint64_t drained;
  unsigned long long total;
  int gave_up;
  uint32_t tmem;
  Item items[kItems];
  float2 stats[2][kRows];
};

// Products and sums of two in one instruction.
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t twice(float x) { return pair_of(__float_as_uint(x), __float_as_uint(x)); }

// cap tanh z, z = scale x / cap, in units of log 2: for |z| <= 0.6 z times a polynomial in z^2
// (fitted to tanh(z) / z by least squares, reweighted until its largest error, 2^-23.7 of the
// value, is about even), else cap (1 - 2 / (1 + e^2z)), within 2^-20 of the value there.  (z itself
// costs a product.  Coefficients for powers of x would save it, but are no 32-bit numbers for large
// caps, and for those the other form is good for nothing: 1 - 2 / (1 + e^2z) is 0 where z is below 2^-24.)
__device__ __forceinline__ float capped(const Params& P, float x) {
  const float z = x * P.cap_unit, u = z * z;
  const float near = z * fmaf(u, fmaf(u, fmaf(u, fmaf(u, P.cap_poly[4], P.cap_poly[3]), P.cap_poly[2]),
                                      P.cap_poly[1]), P.cap_poly[0]);
  const float far = fmaf(rcp_of(exp2_of(z * 2.8853900817779268f) + 1.0f), -2.0f * P.cap_log2, P.cap_log2);
  return fabsf(x) <= P.cap_small ? near : far;
}

// Half a tile's products become capped scores.  Those of a warp's rows rarely leave the
// polynomial, which is seven instructions for two of them; where they do, both forms are taken.
__device__ __forceinline__ void cap_scores(const Params& P, uint32_t (&x)[kHalf]) {
  float most[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int e = 0; e < kHalf; e += 2)
    most[e / 2 % 4] = fmaxf(fmaxf(most[e / 2 % 4], fabsf(__uint_as_float(x[e]))), fabsf(__uint_as_float(x[e + 1])));
  const float all = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
  if (__all_sync(kFullMask, all <= P.cap_small)) {
    const uint64_t k[5] = {twice(P.cap_poly[0]), twice(P.cap_poly[1]), twice(P.cap_poly[2]),
                           twice(P.cap_poly[3]), twice(P.cap_poly[4])};
    const uint64_t unit = twice(P.cap_unit);
#pragma unroll
    for (int e = 0; e < kHalf; e += 2) {
      const uint64_t z = mul2(pair_of(x[e], x[e + 1]), unit), u = mul2(z, z);
      const float2 y = halves_of(mul2(z, fma2(u, fma2(u, fma2(u, fma2(u, k[4], k[3]), k[2]), k[1]), k[0])));
      x[e] = __float_as_uint(y.x);
      x[e + 1] = __float_as_uint(y.y);
    }
  } else {
#pragma unroll
    for (int e = 0; e < kHalf; e++) x[e] = __float_as_uint(capped(P, __uint_as_float(x[e])));
  }
}

// What is done to scores besides their scale: nothing, a cap, a bias (with or without a cap).
enum { kPlain, kCapped, kBiased };

template <class E, int DP, int kMod>
__global__ void __launch_bounds__(kThreads, 1)
    attention_kernel(const Params P, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map) {
  using S = Shape<DP>;
  constexpr int kStages = S::kStages;
  // weights in f16 go below 2^-14, where its steps stop shrinking: taken 2^7 larger
  // they reach 2^15 at most (2^kRise more than the maximum's)
  constexpr float kLift = std::is_same<E, F16>::value ? 7.0f : 0.0f;
  constexpr uint32_t kExp = std::is_same<E, Bf16>::value ? 0x7f80u : 0x7c00u;
  extern __shared__ __align__(1024) char smem[];
  Tail<kStages>& s = *reinterpret_cast<Tail<kStages>*>(smem + S::kTailAt);
  int64_t* const units_at = reinterpret_cast<int64_t*>(smem + S::kStageAt);  // until the copies begin
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  const uint32_t base = smem_of(smem);
  const Cache& C = P.cache;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    for (int i = 0; i < kStages; i++) {
      barrier_init(smem_of(&s.kv_full[i]), P.box_rows ? 1 : 32 * kLoadWarps);
      barrier_init(smem_of(&s.kv_clean[i]), 2);
      barrier_init(smem_of(&s.kv_empty[i]), 4);  // both streams' MMAs, both warps that look at it
    }
    for (int i = 0; i < 2; i++) {
      barrier_init(smem_of(&s.q_full[i]), 32 * kLoadWarps);
      barrier_init(smem_of(&s.q_empty[i]), 2);
      for (int k = 0; k < 2; k++) {
        barrier_init(smem_of(&s.s_full[i][k]), 1);
        barrier_init(smem_of(&s.p_full[i][k]), 4);
        barrier_init(smem_of(&s.o_full[i][k]), 1);
      }
    }
    barrier_init(smem_of(&s.joined), 8);
    barrier_init(smem_of(&s.parted), 8);
    for (int i = 0; i < kItems; i++) {
      barrier_init(smem_of(&s.item_full[i]), 1);
      barrier_init(smem_of(&s.item_checked[i]), 1);
      barrier_init(smem_of(&s.item_empty[i]), kLoadWarps + 4 + 1 + 2 + 8);
    }
    barrier_init(smem_of(&s.drained), 4);
    s.gave_up = 0;
    s.total = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid == 32 * kLoadWarp && P.box_rows) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&k_map) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&v_map) : "memory");
  }
  if (warp == kScoreWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_of(&s.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  // A key head's units of every request: of one row tile by a thread, of more by a warp.
  for (int b = tid; b < P.B; b += kThreads) {
    const Request r = request_of(P, b);
    const int R = row_tiles_of(P, r);
    units_at[b] = R == 0 ? 0 : R == 1 ? units_of(span_of(P, r, 0)) : -1;
  }
  __syncthreads();
  int64_t mine = 0;
  for (int b = warp; b < P.B; b += kThreads / 32) {
    int64_t units = units_at[b];
    if (units < 0) {
      units = head_units(P, request_of(P, b), lane);
      __syncwarp();
      if (lane == 0) units_at[b] = units;
    }
    mine += units;
  }
  if (lane == 0 && mine) atomicAdd(&s.total, static_cast<unsigned long long>(mine) * C.heads);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  // The request in which this run begins, and the units before it.
  const Runs runs(P, static_cast<int64_t>(s.total));
  const int run = blockIdx.x;
  int list_b = 0;
  int64_t list_before = 0;
  if (warp == kListWarp) {
    const int64_t u = runs.start(run);
    while (list_b < P.B) {
      const int64_t units = list_b + lane < P.B ? units_at[list_b + lane] * C.heads : 0;
      int64_t upto = units;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int64_t x = __shfl_up_sync(kFullMask, upto, o);
        if (lane >= o) upto += x;
      }
      const uint32_t past = __ballot_sync(kFullMask, list_before + upto > u);
      if (past) {
        const int from = __ffs(past) - 1;
        list_before += __shfl_sync(kFullMask, upto - units, from);
        list_b += from;
        break;
      }
      list_before += __shfl_sync(kFullMask, upto, 31);
      list_b += 32;
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // tensor copies will write there
  __syncthreads();
  const uint32_t tmem = s.tmem;
  const uint32_t tS[2] = {tmem, tmem + 128};
  const uint32_t tO[2] = {tmem + 256, tmem + 256 + DP};
  volatile int* gave_up = &s.gave_up;
  // The next item of this thread's warp; lane 0 gives it back when it is done.
  uint32_t items = 0;
  auto next_item = [&]() -> const Item& {
    const uint32_t slot = items % kItems;
    barrier_wait(smem_of(&s.item_full[slot]), items / kItems & 1, gave_up);
    return s.items[slot];
  };
  auto done_item = [&]() {
    if (lane == 0) barrier_arrive(smem_of(&s.item_empty[items % kItems]));
    items++;
  };
  auto over = [&](const Item& w) { return w.t0 < 0 || *gave_up; };

  if (warp >= kLoadWarp && warp < kLoadWarp + kLoadWarps) {
    // ------------------------------------------------------------- copies
    asm volatile("setmaxnreg.dec.sync.aligned.u32 " SPECV_CHUNK_REGS_LOAD ";");
    // Copies of 16 bytes, so that pages of any size and strides of any kind will
    // do; places without a key (behind the last, past the head) become 0.
    constexpr int kPieces = DP / 8;            // 16-byte pieces of a row
    constexpr int kRowsAtOnce = 32 / kPieces;  // rows of one warp instruction
    const int lw = warp - kLoadWarp, piece = lane % kPieces, sub = lane / kPieces;
    const bool inside = piece * 8 < C.head_dim;
    uint32_t jobs = 0;  // before this item
    uint32_t sent = 0;  // ... and by tensor copies so far
    uint32_t queries = 0;  // tiles of queries so far
    // 128-byte rows, their 16-byte pieces swapped by the row's number: rows
    // kRowsAtOnce apart, and sub < kRowsAtOnce, so r and sub set bits of their own
    const uint32_t swap = (piece % 8) ^ sub;
    auto tile_copy = [&](uint32_t to, const uint16_t* from, int64_t off) {
      // this lane's row is 32 lw + lane of the tile, at from + off (off < 0: none)
      const uint32_t lane_at = (piece / 8) * (kRows * 128) + (32 * lw + sub) * 128;
#pragma unroll
      for (int r = 0; r < 32; r += kRowsAtOnce) {
        const int64_t o = __shfl_sync(kFullMask, off, r + sub);
        const bool ok = o >= 0 && inside;
        copy16(to + lane_at + r * 128 + (swap ^ (r % 8)) * 16, from + (ok ? o + piece * 8 : 0), ok);
      }
    };
    while (true) {
      const Item& w = next_item();
      if (__any_sync(kFullMask, over(w))) break;
      const bool pair = w.rows > kRows;
      bool going = true;  // the same on every lane
      for (int half = 0; half < (pair ? 2 : 1) && going; half++, queries++) {
        const uint32_t buffer = queries & 1;
        going = __all_sync(kFullMask, barrier_wait(smem_of(&s.q_empty[buffer]), (queries / 2 & 1) ^ 1, gave_up));
        if (!going) break;
        const int row = half * kRows + 32 * lw + lane;
        const bool real = row < w.rows;
        const int at = w.row_tile * kRowTile + (real ? row : 0);
        const int token = at / P.group, g = at - token * P.group;
        const int64_t off = (w.first + static_cast<int64_t>(token)) * P.q.node_stride +
                            (w.h * P.group + g) * P.q.head_stride;
        tile_copy(base + buffer * S::kQueryBytes, P.q.data, real ? off : -1);
        copies_arrive(smem_of(&s.q_full[buffer]));
      }
      if (!going) break;
      // Slots that some row of the item sees; the pages of others are not followed.
      const Keys keys(w);
      const int low = keys.low0, high = max(keys.pos1 + 1, keys.prefix), tiles = keys.tiles;
      const int32_t* table = C.page_table + static_cast<int64_t>(w.b) * C.table_stride;
      // Page numbers are read a tile ahead of their use; one out of range (its
      // request is flagged elsewhere) is no page.  Of keys key .. key+count-1, of one page:
      auto page_at = [&](int key, int count) {
        int page = -1;
        if (key < high && (key < keys.prefix || key + count > low)) page = table[key / C.page_size];
        return page < C.pages ? page : -1;
      };
      if (P.box_rows) {
        // Tensor copies: lane l < boxes brings box l % per_half of 64-column half
        // l / per_half.  A page's rows that nobody sees come along; the
        // softmax clears their values.
        if (lw == kLoadWarps - 1) {
          const int per_half = kKeys / P.box_rows, boxes = per_half * (DP / 64);
          const int box = lane % per_half, half = lane / per_half;
          const int at = box * P.box_rows;
          auto page_of = [&](int i) {
            return i < tiles && lane < boxes ? page_at(keys.first(i) + at, P.box_rows) : -1;
          };
          int page = page_of(0), page_next = page_of(1);
          auto copy = [&](uint32_t job, const CUtensorMap* map, int page, int i) {
            const uint32_t stage = (jobs + job) % kStages, use = (jobs + job) / kStages;
            const uint32_t bar = smem_of(&s.kv_full[stage]);
            const int count = __popc(__ballot_sync(kFullMask, page >= 0));
            if (!__all_sync(kFullMask, barrier_wait(smem_of(&s.kv_empty[stage]), (use & 1) ^ 1, gave_up)))
              return false;
            sent = jobs + job + 1;
            if (lane == 0) barrier_expect(bar, count * P.box_rows * 128);
            __syncwarp();
            if (page >= 0)
              tensor_copy(base + S::kStageAt + stage * S::kTileBytes + half * (kKeys * 128) + at * 128,
                          map, half * 64, (keys.first(i) + at) % C.page_size, w.h, page, bar);
            return true;
          };
          int page_before = -1;
          for (int i = 0; i < tiles && going; i++) {
            going = copy(S::key_job(i), &k_map, page, i);
            if (going && i > 0) going = copy(S::value_job(i - 1, tiles), &v_map, page_before, i - 1);
            page_before = page;
            page = page_next;
            page_next = page_of(i + 2);
          }
          if (going) going = copy(S::value_job(tiles - 1, tiles), &v_map, page_before, tiles - 1);
        }
      } else {
        auto key_of = [&](int i) { return keys.first(i) + 32 * lw + lane; };
        auto page_of = [&](int i) { return i < tiles ? page_at(key_of(i), 1) : -1; };
        int page = page_of(0), page_next = page_of(1);
        auto copy = [&](uint32_t job, const uint16_t* from, int64_t off) {
          const uint32_t stage = (jobs + job) % kStages, use = (jobs + job) / kStages;
          if (!__all_sync(kFullMask, barrier_wait(smem_of(&s.kv_empty[stage]), (use & 1) ^ 1, gave_up)))
            return false;
          tile_copy(base + S::kStageAt + stage * S::kTileBytes, from, off);
          copies_arrive(smem_of(&s.kv_full[stage]));
          return true;
        };
        int64_t before = -1;
        for (int i = 0; i < tiles && going; i++) {
          const int64_t off = page < 0 ? static_cast<int64_t>(-1)
                                       : page * C.page_stride +
                                             key_of(i) % C.page_size * C.row_stride +
                                             w.h * C.head_stride;
          page = page_next;
          page_next = page_of(i + 2);
          going = copy(S::key_job(i), C.k, off);
          if (going && i > 0) going = copy(S::value_job(i - 1, tiles), C.v, before);
          before = off;
        }
        if (going) going = copy(S::value_job(tiles - 1, tiles), C.v, before);
      }
      if (!going) break;
      jobs += 2 * tiles;
      __syncwarp();
      done_item();
    }
    // Copies still in flight, and the arrivals that follow them, must find this CTA's
    // shared memory.  (Where all went well, who reads them waits for them.)
    asm volatile("cp.async.wait_all;" ::: "memory");
    for (uint32_t k = sent < kStages ? 0 : sent - kStages; k < sent; k++)
      barrier_wait_own(smem_of(&s.kv_full[k % kStages]), k / kStages & 1);
    if (*gave_up) {
      const uint64_t start = now_ns();
      while (now_ns() - start < 100000) {
      }
    }
  } else if (warp >= kScoreWarp && warp < kScoreWarp + 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 " SPECV_CHUNK_REGS_OTHER ";");
    // --------------------------------------------------------------- MMAs
    constexpr uint32_t kType = std::is_same<E, Bf16>::value ? 1 : 0;
    constexpr uint32_t kIdesc = 1u << 4 | kType << 7 | kType << 10 | (kRows >> 4) << 24;
    constexpr uint32_t kIdescS = kIdesc | (kHalf >> 3) << 17;
    // Two threads a stream, that neither waits for what the other issues: scores of half a
    // tile when the sum over its stream's last but one has left its place, sums when the
    // weights are there.
    // (A whole warp goes through the loops, on values that the compiler knows to be the same in
    // every lane, and one lane issues: so descriptors are in uniform registers, where a lane
    // by itself would move each there, 100 cycles an MMA.)
    const bool scores = __shfl_sync(kFullMask, warp, 0) < kSumWarp;
    const int st = __shfl_sync(kFullMask, warp, 0) & 1;
    const int steps = (C.head_dim + 15) / 16;
    const uint32_t idesc_sum = kIdesc | 1u << 16 | static_cast<uint32_t>(2 * steps) << 17;
    const uint32_t tm = __shfl_sync(kFullMask, tmem, 0);
    const uint32_t out = tm + 256 + st * DP, place0 = tm + st * 128;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(kFullMask, barrier_wait(smem_of(bar), parity, gave_up)) != 0;
    };
    uint32_t jobs = 0;     // copies before this item
    uint32_t issued = 0;   // halves so far
    uint32_t queries = 0;  // tiles of queries before this item
    while (true) {
      const Item& w = next_item();
      if (__any_sync(kFullMask, over(w))) break;
      Keys keys(w);
      keys.same();
      const Halves halves(keys, __shfl_sync(kFullMask, w.t0, 0));
      const bool pair = __shfl_sync(kFullMask, w.rows, 0) > kRows;
      __syncwarp();
      done_item();
      bool going = true, first = true;
      uint32_t q_at = base;
      if (scores) {
        // (Both streams' warps wait for all of an item's tiles and give all back.  One that waited for
        // its own alone could go through a short item and give a tile back before it was even
        // loaded, for the other's warp.)
        for (uint32_t tile = queries; tile < queries + (pair ? 2 : 1) && going; tile++)
          going = wait(&s.q_full[tile & 1], tile / 2 & 1);
        if (!going) break;
        q_at += ((queries + (pair ? st : 0)) & 1) * S::kQueryBytes;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      uint32_t stage = 0, stage_at = 0;
      int tile = -1, tiles = 0;
      for (int i = 0; i < halves.total; i++) {
        const int key0 = halves.key(i);
        if (key0 / kKeys != tile) {  // the next tile
          if (tiles && elect_one()) mma_commit(smem_of(&s.kv_empty[stage]));
          __syncwarp();
          tile = key0 / kKeys;
          const uint32_t job = jobs + (scores ? S::key_job(tiles) : S::value_job(tiles, keys.tiles));
          tiles++;
          stage = job % kStages;
          stage_at = base + S::kStageAt + stage * S::kTileBytes;
          going = wait(scores ? &s.kv_full[stage] : &s.kv_clean[stage], job / kStages & 1);
          if (!going) break;
          // copies of 16 bytes wrote through the generic proxy, the MMA reads through the other
          if (!P.box_rows) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        if (!pair && (i & 1) != st) continue;  // (of one row tile the streams take halves in turn)
        const uint32_t place = issued & 1, use = issued / 2;
        const uint32_t at = place0 + place * kHalf, from = stage_at + (key0 & kHalf) * 128;
        going = scores ? wait(&s.o_full[st][place], (use & 1) ^ 1) : wait(&s.p_full[st][place], use & 1);
        if (!going) break;
        tmem_fence_after();
        if (scores) {
          const uint32_t a = operand_low(q_at, 16), b = operand_low(from, 16);
          if (elect_one()) {
            mma_ss<false>(at, a, b, kIdescS);
#pragma unroll
            for (int k = 1; k < DP / 16; k++) {
              const uint32_t step = ((k / 4) * (kKeys * 128) + (k % 4) * 32) >> 4;  // of both
              if (k < steps) mma_ss<true>(at, a + step, b + step, kIdescS);
            }
            mma_commit(smem_of(&s.s_full[st][place]));
          }
        } else {
          const uint32_t b = operand_low(from, kKeys * 128);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kHalf / 16; k++)
              mma_ts(out, at + 8 * k, b + (k * 2048 >> 4), idesc_sum, k > 0 || !first);
            mma_commit(smem_of(&s.o_full[st][place]));
          }
          first = false;
        }
        __syncwarp();
        issued++;
      }
      if (!going) break;
      if (elect_one()) mma_commit(smem_of(&s.kv_empty[stage]));
      __syncwarp();
      jobs += 2 * keys.tiles;
      for (int half = 0; half < (pair ? 2 : 1); half++, queries++)
        if (scores && elect_one()) mma_commit(smem_of(&s.q_empty[queries & 1]));
      __syncwarp();
    }
    // every MMA and every arrival that waits for one must find this CTA's memory
    if (elect_one()) {
      mma_commit(smem_of(&s.drained));
      barrier_wait_own(smem_of(&s.drained), 0);
    }
    __syncwarp();
  } else if (warp >= kListWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 " SPECV_CHUNK_REGS_OTHER ";");
    // ------------------------------------------------------------ listing
    if (warp == kListWarp) {
      int b = list_b;
      int64_t before = list_before;
      bool stop = false, begins = true;
      // every run's, whatever is in it: the join follows what it finds
      if (lane == 0) P.ws.cuts[run] = Cut{0, 0, 0, 0, 0, 0, 0, 0};
      int64_t u = runs.start(run);
      const int64_t end = runs.start(run + 1);
      while (u < end && b < P.B && !stop) {
        const Request r = request_of(P, b);
        const int64_t head = head_units(P, r, lane);
        const int R = row_tiles_of(P, r);
        while (u < end && u < before + head * C.heads) {
          const int h = static_cast<int>(Runs::quotient(u - before, head));
          const int64_t off = u - before - h * head;
          // the row tile with this unit: 32 of them at a time
          int row_tile = 0;
          int64_t passed = 0;
          Span span;
          int units;
          while (true) {
            units = 0;
            if (row_tile + lane < R) {
              span = span_of(P, r, row_tile + lane);
              units = units_of(span);
            }
            int64_t upto = units;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
              const int64_t x = __shfl_up_sync(kFullMask, upto, o);
              if (lane >= o) upto += x;
            }
            const uint32_t past = __ballot_sync(kFullMask, passed + upto > off);
            if (past) {
              const int from = __ffs(past) - 1;
              passed += __shfl_sync(kFullMask, upto - units, from);
              row_tile += from;
              break;
            }
            passed += __shfl_sync(kFullMask, upto, 31);
            row_tile += 32;
            if (row_tile >= R) {  // the lengths changed meanwhile
              stop = true;
              break;
            }
          }
          if (stop) break;
          span = span_of(P, r, row_tile);
          const int weight = span.rows > kRows ? 2 : 1;
          // its first tile's first unit, and what of its tiles this run has
          const int64_t first = before + h * head + passed + cost_of(span);
          auto tile_of = [&](int64_t unit) {
            return static_cast<int>(min(max(unit - first + weight - 1, static_cast<int64_t>(0)) / weight,
                                        static_cast<int64_t>(span.tiles)));
          };
          const int t0 = tile_of(u), t1 = tile_of(end);
          u = min(end, first + weight * span.tiles);
          if (t1 <= t0) continue;  // the run ends before the item's first tile
          // runs before and behind with pieces of this item
          int first_run = run, last_run = run;
          if (t0 > 0) first_run = runs.of(first);
          if (t1 < span.tiles) last_run = runs.of(first + weight * (span.tiles - 1));
          const uint32_t slot = items % kItems;
          barrier_wait(smem_of(&s.item_empty[slot]), (items / kItems & 1) ^ 1, gave_up);
          stop = __any_sync(kFullMask, *gave_up != 0);
          if (stop) break;
          if (lane == 0) {
            const int pieces = last_run - first_run + 1;
            s.items[slot] = Item{b, h, row_tile, t0, t1, span.gap, span.skip, span.rows, r.first, r.n,
                                 r.len, r.prefix, span.pos0, span.pos1, lowest(P, span.pos0),
                                 lowest(P, span.pos1), pieces, t0 == 0, 0, 0, {}};
            if (begins && t0 > 0 && first_run == run - 1)
              P.ws.cuts[run] = Cut{b, h, row_tile, span.rows, r.first, pieces, 0, 0};
          }
          __syncwarp();
          if (lane == 0) barrier_arrive(smem_of(&s.item_full[slot]));
          items++;
          begins = false;
        }
        before += head * C.heads;
        b++;
      }
      {
        const uint32_t slot = items % kItems;
        barrier_wait(smem_of(&s.item_empty[slot]), (items / kItems & 1) ^ 1, gave_up);
        if (lane == 0 && !*gave_up) {
          s.items[slot].t0 = -1;
          barrier_arrive(smem_of(&s.item_full[slot]));
        }
      }
    }
    // ----------------------------------------------------------- checking
    // This CTA's share of all requests for their status, and every item's
    // request for what its rows become, whenever an item is there.
    if (warp == kCheckWarp) {
      auto check = [&](int b, Request& r) {
        r = request_of(P, b);
        if (!r.bad && r.n &&
            __any_sync(kFullMask, bad_pages(C, b, 0, r.prefix, lane, 32) ||
                                      bad_pages(C, b, lowest(P, r.len), r.len + r.n, lane, 32)))
          r.bad |= SPECV_DEV_BAD_CACHE;
        return r.bad;
      };
      int next = blockIdx.x, last = -1, last_bad = 0;
      Request r;
      auto report = [&]() {
        const unsigned bad = check(next, r);
        if (lane == 0) P.status[next] = static_cast<int32_t>(bad);
        if (bad && row_tiles_of(P, request_of(P, next)) == 0) {  // no item has its rows
          const int words = C.head_dim / 8;
          const int64_t all = static_cast<int64_t>(r.n) * P.q_heads * words;
          for (int64_t e = lane; e < all; e += 32) {
            const int64_t i = e / (P.q_heads * words);
            const int left = static_cast<int>(e - i * (P.q_heads * words)), h = left / words, d = left % words * 8;
            *reinterpret_cast<uint4*>(P.out.data + (r.first + i) * P.out.node_stride +
                                      h * P.out.head_stride + d) = make_uint4(0, 0, 0, 0);
          }
        }
        next += gridDim.x;
      };
      while (true) {
        const uint32_t slot = items % kItems;
        if (next < P.B &&
            !__any_sync(kFullMask, barrier_test(smem_of(&s.item_full[slot]), items / kItems & 1))) {
          report();
          continue;
        }
        Item& w = s.items[slot];
        barrier_wait(smem_of(&s.item_full[slot]), items / kItems & 1, gave_up);
        if (__any_sync(kFullMask, over(w))) {
          while (next < P.B) report();
          break;
        }
        if (w.b != last) last_bad = static_cast<int>(check(w.b, r));
        last = w.b;
        if (lane == 0) w.bad = last_bad;
        __syncwarp();
        if (lane == 0) barrier_arrive(smem_of(&s.item_checked[slot]));
        done_item();
      }
    }
    // ------------------------------------------------- values not all rows see
    // A value that is not finite would pass through a weight of 0 into rows that do
    // not see its key: it becomes 0 here and comes back, at the end, for those that do.
    // (And what lies where nobody sees a key is whatever was there.)
    if (warp >= kCleanWarp) {
      uint32_t jobs = 0;
      auto pass = [&](uint32_t job, auto clean) {
        const uint32_t stage = job % kStages;
        if (!__all_sync(kFullMask, barrier_wait(smem_of(&s.kv_full[stage]), job / kStages & 1, gave_up)))
          return false;
        clean(smem + S::kStageAt + stage * S::kTileBytes);
        __syncwarp();
        if (lane == 0) {
          barrier_arrive(smem_of(&s.kv_clean[stage]));
          barrier_arrive(smem_of(&s.kv_empty[stage]));
        }
        return true;
      };
      auto look = [](char*) {};
      while (true) {
        Item& w = const_cast<Item&>(next_item());
        if (__any_sync(kFullMask, over(w))) break;
        const Keys keys(w);
        bool going = true;
        auto values = [&](int i) {
          const int tile_key = keys.first(i);
          return pass(jobs + S::value_job(i, keys.tiles), [&](char* v) {
            if (!keys.mixed(tile_key, kKeys)) return;
            constexpr int kPieces = DP / 8;  // of a row
            const int me = (warp - kCleanWarp) * 32 + lane, piece = me % kPieces;
            char* const column = v + (piece / 8) * (kKeys * 128) + (piece % 8) * 16;
            // rows [from, to) of the tile, as keys; those below the prefix are seen by all
            auto rows = [&](int from, int to, auto each) {
              const int last = min(to - tile_key, kKeys);
              for (int r = max(max(from, keys.prefix) - tile_key, 0) + me / kPieces; r < last; r += 64 / kPieces)
                each(r, reinterpret_cast<uint4*>(column + r * 128));
            };
            auto clear = [](int, uint4* place) { *place = make_uint4(0, 0, 0, 0); };
            auto check = [&](int r, uint4* place) {
              // the exponent's bits, and one of its lowest more: the top bit where all are set
              constexpr uint32_t kBits = kExp * 0x10001u, kLowest = (kExp & (0u - kExp)) * 0x10001u;
              uint4 x = *place;
              uint32_t* words = &x.x;
              uint32_t odd[4];
#pragma unroll
              for (int i = 0; i < 4; i++) odd[i] = ((words[i] & kBits) + kLowest) & 0x80008000u;
              if (!(odd[0] | odd[1] | odd[2] | odd[3])) return;
#pragma unroll
              for (int i = 0; i < 4; i++) words[i] &= ~((odd[i] >> 15) * 0xffffu);
              *place = x;
              const int key = tile_key + r;
              const int bit = key > keys.pos0 ? key - keys.pos0 - 1 : 32 * kEdge + key - keys.low0;
              atomicOr(w.odd + bit / 32, 1u << bit % 32);
              w.any_odd = 1;
            };
            rows(tile_key, keys.low0, clear);  // nobody sees them
            rows(keys.low0, min(keys.low1, keys.pos0 + 1), check);
            rows(max(keys.low0, keys.pos0 + 1), keys.pos1 + 1, check);
            rows(keys.pos1 + 1, tile_key + kKeys, clear);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          });
        };
        for (int i = 0; i < keys.tiles && going; i++) {
          going = pass(jobs + S::key_job(i), look);
          if (going && i > 0) going = values(i - 1);
        }
        if (going) going = values(keys.tiles - 1);
        if (!going) break;
        jobs += 2 * keys.tiles;
        __syncwarp();
        done_item();
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 " SPECV_CHUNK_REGS_SOFTMAX ";");
    const int st = warp / 4, quarter = warp % 4;
    const int row = quarter * 32 + lane;  // of the stream's tile
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    uint32_t scored = 0;  // halves of tiles of this stream so far
    uint32_t shared = 0;            // items that both streams had parts of
    while (true) {
      Item& w = const_cast<Item&>(next_item());
      if (__any_sync(kFullMask, over(w))) break;
      const bool pair = w.rows > kRows;
      const int first_row = pair ? st * kRows : 0, rows = w.rows;
      const bool working = first_row + quarter * 32 < rows;  // this warp has rows
      const int at = w.row_tile * kRowTile + min(first_row + row, rows - 1);
      const int token = at / P.group, g = at - token * P.group;
      // slots that this row sees: below the prefix, and low .. pos
      const Keys keys(w);
      const int pos = w.len + token, low = lowest(P, pos), prefix = keys.prefix;
      const float slope = kMod && P.slopes ? P.slopes[w.h * P.group + g] * 1.4426950408889634f : 0.0f;
      int taken = 0;  // halves of this item that this stream took
      float m = -INFINITY, l = 0.0f;  // m: the maximum that O and l were taken with

      const Halves halves(keys, w.t0);
#pragma unroll 1
      for (int i = pair ? 0 : st; i < halves.total; i += pair ? 1 : 2) {
        // (of an item of one row tile the streams take halves in turn)
        const int key0 = halves.key(i);
        const uint32_t place = scored & 1, use = scored / 2;
        if (!__all_sync(kFullMask, barrier_wait(smem_of(&s.s_full[st][place]), use & 1, gave_up))) break;
        __syncwarp();  // (lanes may leave a wait apart, and tensor memory is read by whole warps)
        tmem_fence_after();
        const bool first = taken++ == 0;
        bool going = true;  // the same on every lane
        if (working) {
          const uint32_t at_s = tS[st] + lanes + place * kHalf;
          uint32_t x[kHalf];
          tmem_load64(at_s, x);
          // A score is mult x + base + step e in units of log 2, for the half's e-th key.
          float mult = P.scale_log2, base = 0.0f, step = 0.0f;
          if (kMod && P.cap_log2 > 0.0f) {
            cap_scores(P, x);
            mult = 1.0f;
          }
          if (kMod == kBiased) {
            if (key0 + kHalf - 1 <= keys.pos0) {  // no key is in front of a row
              base = slope * static_cast<float>(key0 - pos);
              step = slope;
            } else {
#pragma unroll
              for (int e = 0; e < kHalf; e++)
                x[e] = __float_as_uint(fmaf(-slope, fabsf(static_cast<float>(key0 - pos + e)),
                                            __uint_as_float(x[e]) * mult));
              mult = 1.0f;
            }
          }
          if (keys.mixed(key0, kHalf)) {
#pragma unroll
            for (int k = 0; k < kHalf; k += 32) {
              const int from = key0 + k;
              const uint32_t seen =
                  bits_below(prefix - from) | (bits_below(pos + 1 - from) & ~bits_below(low - from));
#pragma unroll
              for (int e = 0; e < 32; e++)
                if (!(seen >> e & 1)) x[k + e] = 0xff800000u;  // -inf
            }
          }
          // The weights with the maximum so far, beside the half's own: where that is too much
          // above it, once more.
          const uint64_t mult2 = twice(mult);
          uint32_t p[kHalf / 2];
          float sum;
          bool again = false;
#pragma unroll 1
          while (true) {
            const float shift = kLift - (m == -INFINITY ? 0.0f : m);
            const float from = base + shift;
            const uint64_t shift2 = twice(shift);
            uint64_t sums[2] = {0, 0};
            float tops[4];
#pragma unroll
            for (int e = 0; e < kHalf; e += 2) {
              const uint64_t xs = pair_of(x[e], x[e + 1]);
              uint64_t y2;
              if (kMod == kPlain) {
                y2 = fma2(xs, mult2, shift2);
              } else if (kMod == kCapped) {
                y2 = add2(xs, shift2);
              } else {
                const float lo = fmaf(step, static_cast<float>(e), from), hi = fmaf(step, static_cast<float>(e + 1), from);
                y2 = fma2(xs, mult2, pair_of(__float_as_uint(lo), __float_as_uint(hi)));
              }
              const float2 y = halves_of(y2);
              const float a = exp2_of(y.x), b = exp2_of(y.y);
              // (the largest of what costs least to have: products, or scores less the shift)
              const float u = kMod == kBiased ? y.x : __uint_as_float(x[e]);
              const float v = kMod == kBiased ? y.y : __uint_as_float(x[e + 1]);
              tops[e / 2 % 4] = e < 8 ? fmaxf(u, v) : max3(tops[e / 2 % 4], u, v);
              sums[e / 2 % 2] = add2(sums[e / 2 % 2], pair_of(__float_as_uint(a), __float_as_uint(b)));
              // the weights' one rounding, to the type of the values they meet: the MMA takes
              // both operands in one 16-bit type.  (The sum has them as they are.)
              p[e / 2] = E::pack(a, b);
            }
            const float2 both = halves_of(add2(sums[0], sums[1]));
            sum = both.x + both.y;
            float top = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]);
            if (kMod == kPlain) top *= mult;
            if (kMod == kBiased) top -= shift;
            const bool rise = first || top > m + kRise;
            if (again || !__any_sync(kFullMask, rise)) break;
            again = true;
            float by = 1.0f;
            if (rise) {
              const float higher = fmaxf(m, top);
              by = higher == -INFINITY ? 1.0f : exp2_of(m - higher);
              m = higher;
            }
            if (!first) {
              // the last update of O must be done
              const uint32_t last = scored - 1;
              going = __all_sync(kFullMask, barrier_wait(smem_of(&s.o_full[st][last & 1]), last / 2 & 1, gave_up));
              if (!going) break;
              __syncwarp();
              tmem_fence_after();
              l *= by;
#pragma unroll 1
              for (int k = 0; k < DP; k += 16) {
                uint32_t o[16];
                tmem_load16(tO[st] + lanes + k, o);
#pragma unroll
                for (int e = 0; e < 16; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * by);
                tmem_store16(tO[st] + lanes + k, o);
              }
            }
          }
          if (!going) break;
          l += sum;
          __syncwarp();
          tmem_store32(at_s, p);  // over scores of this row, all read
          tmem_store_wait();
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) barrier_arrive(smem_of(&s.p_full[st][place]));
        scored++;
      }

      // The item's end: this stream's last sum, and where both have parts of the rows the
      // other's too.  (Whichever of these waits gave up, in whichever lane, `bad` says so in all of them:
      // then neither the other's numbers nor tensor memory are read, for they may not be there.)
      if (taken) {
        const uint32_t last = scored - 1;
        barrier_wait(smem_of(&s.o_full[st][last & 1]), last / 2 & 1, gave_up);
      }
      if (!pair) {
        s.stats[st][row] = make_float2(m, l);
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) barrier_arrive(smem_of(&s.joined));
        barrier_wait(smem_of(&s.joined), shared & 1, gave_up);
      }
      tmem_fence_after();
      barrier_wait(smem_of(&s.item_checked[items % kItems]), items / kItems & 1, gave_up);
      const bool bad = __any_sync(kFullMask, w.bad != 0 || *gave_up);  // unchecked is bad
      __syncwarp();
      // A pair: this stream's rows, all columns; else half of the columns of both streams' sum
      const int my_rows = rows - first_row;
      if (quarter * 32 < my_rows && !(bad && !w.begins)) {
        float weight[2] = {1.0f, 1.0f};
        const bool took[2] = {halves.summed(pair, st, 0, bad), halves.summed(pair, st, 1, bad)};
        if (!pair && !bad) {
          const float2 other = s.stats[st ^ 1][row];
          const float m_of[2] = {st ? other.x : m, st ? m : other.x};
          const float l_of[2] = {st ? other.y : l, st ? l : other.y};
          m = fmaxf(m_of[0], m_of[1]);
          l = 0.0f;
#pragma unroll
          for (int k = 0; k < 2; k++) {
            weight[k] = !took[k] ? 0.0f : m_of[k] == m ? 1.0f : exp2_of(m_of[k] - m);
            if (took[k]) l += weight[k] * l_of[k];
          }
        }
        // (The code of an item's end is short on purpose: it is fetched anew for each.)
        const bool whole = w.pieces == 1 || bad;  // of a flagged request the first piece clears the rows
        const bool mine = row < my_rows;
        uint16_t* const out = P.out.data + (w.first + static_cast<int64_t>(token)) * P.out.node_stride +
                              (w.h * P.group + g) * P.out.head_stride;
        const int64_t slot = 2 * static_cast<int>(blockIdx.x) + w.begins;
        float4* const part = P.ws.parts + slot * (DP / 4) * P.part_rows + first_row + row;
        const int cols = pair ? DP : DP / 2, col0 = pair ? 0 : st * cols;
        const float inv = whole ? 1.0f / l : 1.0f;
        const int own = lane & 3;
        uint16_t* to[4];  // rows of lanes ^ 0 .. 3
#pragma unroll
        for (int r = 0; r < 4; r++)
          to[r] = reinterpret_cast<uint16_t*>(
              __shfl_xor_sync(kFullMask, reinterpret_cast<uint64_t>(mine ? out : nullptr), r));
#pragma unroll 1
        for (int k = col0; k < col0 + cols; k += 32) {
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; e++) o[e] = 0.0f;
#pragma unroll 1
          for (int i = pair ? st : 0; i <= (pair ? st : 1); i++) {
            uint32_t x[32];
            if (!(i ? took[1] : took[0])) continue;
            const float by = (i ? weight[1] : weight[0]) * inv;
            __syncwarp();
            tmem_load32(tmem + 256 + i * DP + lanes + k, x);
#pragma unroll
            for (int e = 0; e < 32; e++) o[e] = fmaf(__uint_as_float(x[e]), by, o[e]);
          }
          if (whole) {
            uint4 v[4];
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              v[e / 8] = make_uint4(E::pack(o[e], o[e + 1]), E::pack(o[e + 2], o[e + 3]),
                                    E::pack(o[e + 4], o[e + 5]), E::pack(o[e + 6], o[e + 7]));
              if (bad) v[e / 8] = make_uint4(0, 0, 0, 0);
            }
            // Four lanes have four pieces of 16 bytes of four rows: each takes one piece of every
            // row, so that a store has 64 bytes of a row together.
            const int d = k + 8 * own;
#pragma unroll
            for (int r = 0; r < 4; r++) {
              const uint4 lo = (own ^ r) & 1 ? v[1] : v[0], hi = (own ^ r) & 1 ? v[3] : v[2];
              uint4 x = (own ^ r) & 2 ? hi : lo;  // piece own ^ r of this lane's row
              if (r) {
                x.x = __shfl_xor_sync(kFullMask, x.x, r);
                x.y = __shfl_xor_sync(kFullMask, x.y, r);
                x.z = __shfl_xor_sync(kFullMask, x.z, r);
                x.w = __shfl_xor_sync(kFullMask, x.w, r);
              }
              if (to[r] && d < C.head_dim) *reinterpret_cast<uint4*>(to[r] + d) = x;
            }
          } else if (mine) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              part[(k + e) / 4 * P.part_rows] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
          __syncwarp();
        }
        // Values that are not finite come back where they are seen.  Only a checked request's
        // pages are followed.  (Of a flagged one a box may not have been copied, and what its
        // place in the ring held before may look like such values.)
        if (w.any_odd && !bad && mine) {
#pragma unroll 1
          for (int bit = 0; bit < 64 * kEdge; bit++) {
            if (!(w.odd[bit / 32] >> bit % 32 & 1)) continue;
            const int key = bit < 32 * kEdge ? keys.pos0 + 1 + bit : keys.low0 + bit - 32 * kEdge;
            if (key > pos || key < low) continue;
            const uint16_t* v = C.v + C.slot(w.b, key) + w.h * C.head_stride;
#pragma unroll 1
            for (int d = col0; d < min(col0 + cols, C.head_dim); d++) {
              const uint32_t bits = v[d];
              if ((bits & kExp) != kExp) continue;
              const float odd = E::unpack(bits).x;
              if (whole) out[d] = static_cast<uint16_t>(E::pack(E::unpack(out[d]).x + odd, 0.0f));
              else reinterpret_cast<float*>(part + d / 4 * P.part_rows)[d % 4] += odd;
            }
          }
        }
        __syncwarp();
        if (!whole && mine && (pair || st == 0))
          P.ws.stats[slot * P.part_rows + first_row + row] = make_float2(m, l);
      }
      tmem_fence_before();
      __syncwarp();
      done_item();
      if (!pair) {  // the other's sums may be written over when both have read them
        if (lane == 0) barrier_arrive(smem_of(&s.parted));
        barrier_wait(smem_of(&s.parted), shared++ & 1, gave_up);
        tmem_fence_after();
      }
    }
  }

  tmem_fence_before();
  __syncthreads();
  if (tid == 0 && s.gave_up) P.ws.cuts[blockIdx.x].gave_up = 1;
  if (warp == kScoreWarp) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// -------------------------------------------------------------------- join

// Joins the pieces of the items that runs cut:
//   m = max m_i, O = sum 2^(m_i - m) O_i / sum 2^(m_i - m) l_i, in order.
// A block to 16 rows of a run's cut; that of a run that gave up flags the whole call
// (whose statuses are all written by now).  A warp takes eight rows and kJoinPieces
// pieces at a time, all of their loads in flight; the warps of a row group share out the
// pieces.  A lane has one row and every fourth four columns of it.
constexpr int kJoinRows = 8;
constexpr int kJoinWarps = 8, kJoinGroups = 2, kJoinShares = kJoinWarps / kJoinGroups;
constexpr int kJoinPieces = 4;

template <class E, int DP>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const Params P) {
  constexpr int kQuads = DP / 16;  // of a lane
  __shared__ float4 s_o[kJoinWarps][kQuads][32];
  __shared__ float2 s_ml[kJoinWarps][kJoinRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int group = warp % kJoinGroups, share = warp / kJoinGroups;
  const int run = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Cut cut = P.ws.cuts[run];
  if (cut.gave_up && blockIdx.y == 0)
    for (int b = threadIdx.x; b < P.B; b += kJoinWarps * 32) atomicOr(P.status + b, SPECV_DEV_TIMEOUT);
  // (A call that gave up may leave records of another: they are not followed out of bounds.)
  if (cut.pieces < 2 || cut.pieces > P.ctas - run + 1 || cut.b < 0 || cut.b >= P.B || cut.h < 0 ||
      cut.h >= P.cache.heads || cut.rows < 1 || cut.rows > min(kRowTile, P.part_rows) ||
      cut.row_tile < 0 || cut.row_tile > (INT_MAX >> 9) || cut.first < 0 ||
      cut.first + static_cast<int64_t>(cut.row_tile * kRowTile + cut.rows - 1) / P.group >= P.T)
    return;
  const int first = blockIdx.y * (kJoinGroups * kJoinRows);
  if (first >= cut.rows) return;
  const int flagged = P.status[cut.b];  // its first piece has cleared the rows
  const int row = lane % kJoinRows, quad = lane / kJoinRows;
  const int row0 = first + group * kJoinRows;
  // (slots have whole eights of rows)
  const int at = min(row0, P.part_rows - kJoinRows) + row;
  float m = -INFINITY, l = 0.0f;
  float4 o[kQuads];
#pragma unroll
  for (int j = 0; j < kQuads; j++) o[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  // What is there so far keeps `old` of its weight, the other gets `by`.
  auto add = [&](float old, float by, const float4* x, int step) {
#pragma unroll
    for (int j = 0; j < kQuads; j++) {
      const float4 y = x[j * step];
      o[j].x = fmaf(by, y.x, o[j].x * old);
      o[j].y = fmaf(by, y.y, o[j].y * old);
      o[j].z = fmaf(by, y.z, o[j].z * old);
      o[j].w = fmaf(by, y.w, o[j].w * old);
    }
  };
#pragma unroll 1
  for (int i0 = share * kJoinPieces; i0 < cut.pieces; i0 += kJoinShares * kJoinPieces) {
    float4 x[kJoinPieces][kQuads];
    float2 ml[kJoinPieces];
#pragma unroll
    for (int i = 0; i < kJoinPieces; i++) {
      // the first piece ends a run, the others begin theirs
      const int piece = i0 + i;
      const int64_t slot = 2 * (run - 1 + piece) + (piece == 0);
      const bool real = piece < cut.pieces;
      const float4* from = P.ws.parts + (slot * (DP / 4) + quad) * P.part_rows + at;
      ml[i] = real ? P.ws.stats[slot * P.part_rows + at] : make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int j = 0; j < kQuads; j++)
        x[i][j] = real ? from[4 * j * P.part_rows] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    float top = m;
#pragma unroll
    for (int i = 0; i < kJoinPieces; i++) top = fmaxf(top, ml[i].x);
    float old = m == top ? 1.0f : exp2_of(m - top);
    m = top;
#pragma unroll
    for (int i = 0; i < kJoinPieces; i++) {
      const float by = i0 + i >= cut.pieces ? 0.0f : ml[i].x == top ? 1.0f : exp2_of(ml[i].x - top);
      l = fmaf(by, ml[i].y, l * old);
      add(old, by, x[i], 1);
      old = 1.0f;
    }
  }
  // the warps' shares, in their order
  if (quad == 0) s_ml[warp][row] = make_float2(m, l);
#pragma unroll
  for (int j = 0; j < kQuads; j++) s_o[warp][j][lane] = o[j];
  __syncthreads();
  if (share) return;
#pragma unroll 1
  for (int w = 1; w < kJoinShares; w++) {
    const float2 ml = s_ml[warp + w * kJoinGroups][row];
    const float top = fmaxf(m, ml.x);
    const float old = m == top ? 1.0f : exp2_of(m - top);
    const float by = ml.x == top ? 1.0f : exp2_of(ml.x - top);
    m = top;
    l = fmaf(by, ml.y, l * old);
    add(old, by, &s_o[warp + w * kJoinGroups][0][lane], 32);
  }
  if (row0 + row >= cut.rows || flagged) return;
  const float inv = 1.0f / l;
  const int flat = cut.row_tile * kRowTile + row0 + row, token = flat / P.group, g = flat - token * P.group;
  uint16_t* out = P.out.data + (cut.first + static_cast<int64_t>(token)) * P.out.node_stride +
                  (cut.h * P.group + g) * P.out.head_stride;
#pragma unroll
  for (int j = 0; j < kQuads; j++) {
    const int d = 4 * (quad + 4 * j);
    if (d < P.cache.head_dim)
      *reinterpret_cast<uint2*>(out + d) = make_uint2(E::pack(o[j].x * inv, o[j].y * inv),
                                                      E::pack(o[j].z * inv, o[j].w * inv));
  }
}

template <class E, int DP, int kMod>
cudaError_t launch(const Params& P, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream) {
  using S = Shape<DP>;
  constexpr int kSmem = S::kTailAt + static_cast<int>(sizeof(Tail<S::kStages>));
  static_assert(kSmem <= 232448, "one CTA's shared memory");
  cudaError_t e = cudaFuncSetAttribute(attention_kernel<E, DP, kMod>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  attention_kernel<E, DP, kMod><<<P.ctas, kThreads, kSmem, stream>>>(P, k_map, v_map);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(P.ctas, (P.part_rows + kJoinGroups * kJoinRows - 1) / (kJoinGroups * kJoinRows));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<E, DP>, P);
}

// Whether the call is for the small kernel (single.cuh): no request has more than one token, a key
// head no more than 16 rows, and there are few key heads' slots (their lengths are on the device:
// what the page table or the window has room for stands for them).
// The slots of a prefix beside a window are not known here either, and not counted: as a rule they are the few
// first tokens that a window keeps.  With a table of 32,000 slots, a window of 512 and 8 key heads, one, four and
// eight requests take 19, 19, 19 us here and 23, 25, 29 in the other kernel where the prefix has 4
// slots, 66, 130, 234 and 48, 103, 167 where it has 27,000.
inline bool singles(const Params& P) {
  const int64_t heads = static_cast<int64_t>(P.B) * P.cache.heads;
  const int64_t slots = static_cast<int64_t>(P.cache.max_pages) * P.cache.page_size;
  return P.longest == 1 && P.group <= 16 && heads <= kSms / 2 &&
         heads * (slots < P.window ? slots : P.window) <= 65536;
}

// One translation unit for each type of the cache.
template <class E>
cudaError_t run(const Params& P, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream);

template <class E>
cudaError_t run_any(const Params& P, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
  const bool narrow = P.cache.head_dim <= 64;
  if (P.slopes) return narrow ? launch<E, 64, kBiased>(P, k, v, stream) : launch<E, 128, kBiased>(P, k, v, stream);
  if (P.cap_log2 > 0.0f)
    return narrow ? launch<E, 64, kCapped>(P, k, v, stream) : launch<E, 128, kCapped>(P, k, v, stream);
  return narrow ? launch<E, 64, kPlain>(P, k, v, stream) : launch<E, 128, kPlain>(P, k, v, stream);
}

}  // namespace specv_chunk
