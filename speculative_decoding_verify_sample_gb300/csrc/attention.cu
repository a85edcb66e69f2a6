// Attention of a drafted tree's nodes over the paged cache.
//
// For one key head h of one request the query rows are the (node, query head)
// pairs of its group: n * G rows that read the same keys and values.  They
// make the 128 rows of a tensor-core tile, so a cache row is read from HBM
// once for all of them, whatever N and G are:
//
//   S = Q K^T (tcgen05, operands in shared memory, S in TMEM),
//   P = exp2(S c - m c), c = scale log2 e, m the running row maximum,
//   O = O + P V (tcgen05, P from TMEM where S was, V in shared memory),
//
// and O is rescaled only when the maximum has risen by more than 2^8 (a known
// form of the running softmax), which no result shows: m is whatever both O and the
// sum l were taken with.
//
// The work is the list of (request, key head, row tile, 128-key tile), a unit
// each, cut into even runs, one for every CTA (one to an SM), whatever the
// requests' lengths are.  A row tile whose keys one run has whole is written out;
// pieces leave (m, l, O) in the workspace for join_kernel.
//
// Two streams share an SM, each with its S and O in TMEM and its four softmax
// warps: with up to 128 rows they take the key tiles in turn and are joined
// at the end, with more they are two row tiles on the same keys
// (kPair).  Of the other warps four copy, two threads issue the MMAs, one
// warp lists the run's work and one checks the requests' data beside it all.
//
// Up to 128 rows the cache's bytes bound it: a tile of keys and one of values, 64 KB,
// take an SM 1.5 us and their MMAs 0.7.  Measured: eight chains over 16,111 to
// 32,749 keys 134 us (801 MB, 6.0 TB/s), 32 trees over 97 to 4,093 keys 68 us (288 MB,
// 4.2 TB/s: about 8 us until the first scores and 8 for the join are fixed), one
// token over 1,999 keys 16.4 us, nearly all of it such latencies.  With more rows no
// unit is full: 64 nodes of 64 heads over 4,001 to 8,111 keys take 395 to 408 us (1,010
// TFLOP/s; under the profiler tensor pipe 51 % active, tensor memory 53, shared memory's
// banks 19, issue 35, DRAM 60).  What is left is the chain of scores, softmax and
// sum in each stream, of which TMEM holds two.

#include <cuda.h>

#include <type_traits>

#include "cache.cuh"
#include "tensor.cuh"

using namespace specv_cache_ops;
using namespace specv_tensor;

namespace {

constexpr int kKeys = 128;     // keys of a tile
constexpr int kRows = 128;     // query rows of a stream
static_assert(kKeys == kRows, "tiles of queries, keys and values are laid out alike");
constexpr int kMaxCtas = kSms;
constexpr int kLoadWarps = 4;
constexpr int kLoadWarp = 8;  // the first of them; the last makes the tensor copies
constexpr int kCheckWarp = 12;
constexpr int kScoreWarp = 13;  // issues S = Q K^T
constexpr int kSumWarp = 14;    // issues O += P V
constexpr int kListWarp = 15;
constexpr int kThreads = 512;
constexpr int kItems = 4;  // items listed ahead
// What an item takes besides its key tiles, in their time: its end, and the next
// one's first scores (a batch of 32 trees: 90.8, 78.4, 73.5, 70.3, 70.1 us with 0 .. 4;
// 64-node trees 368.6, 365.6, 365.8, 363.8, 368.7).
constexpr int kItemCost = 3;
// Registers a thread of each warpgroup: 2 * 192 + 72 + 56 = 512 = 4 * 128, what
// the block is launched with.  The softmax keeps a row of scores in them.
#define SPECV_REGS_SOFTMAX "192"
#define SPECV_REGS_LOAD "72"
#define SPECV_REGS_OTHER "56"
constexpr float kRise = 8.0f;  // log2 of how far a maximum may rise before O is rescaled

// ---------------------------------------------------------------- the work

// Where a run begins in the middle of an item: the item's second piece.  And
// whether one of the run's waits gave up, so that it may have left items undone.
struct Cut {
  int32_t b, h, row_tile, n;
  int32_t pieces;  // of the item; 0: the run does not begin with an item's second piece
  int32_t gave_up;
  int32_t pad[2];
};

struct Workspace {
  Cut* cuts;      // [runs]
  float2* stats;  // [2 runs][part_rows] pieces' m c and l: of an item that began before the
                  // run, then of one that goes on behind it
  float4* parts;  // [2 runs][dim / 4][part_rows] their O, four columns of a row together: the
                  // softmax's lanes have a row each, and adjacent rows make whole lines
};

struct AttnParams {
  Cache cache;
  Rows q, out;
  Workspace ws;
  const int32_t* parents;
  const int32_t* n_nodes;
  int32_t* status;
  int B, N, q_heads, group;  // group: query heads to a key head
  int ctas;                  // and runs
  int part_rows;             // rows of a piece in the workspace
  int box_rows;              // rows that one tensor copy brings; 0: copies of 16 bytes
  float scale_log2;
};

// How the units are cut into runs.  (A share dealt out to CTAs as they finish evens
// out the ends, but costs pieces written and read: 16 requests of 4,300 keys took
// 88 us against 69, eight of 24,000 148 against 137.)
struct Runs {
  int64_t total, each;

  __device__ __forceinline__ Runs(const AttnParams& P, int64_t units)
      : total(units), each(quotient(units + P.ctas - 1, P.ctas)) {}
  static __device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return (a | b) >> 32 ? a / b : static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  }
  // Where run `run` begins, and run - 1 ends.
  __device__ __forceinline__ int64_t start(int run) const { return min(total, run * each); }
  // The run that has unit u.
  __device__ __forceinline__ int of(int64_t u) const { return static_cast<int>(quotient(u, each)); }
};

// Nodes of request b, 0 where its count or length is out of range.
__device__ __forceinline__ int nodes_of(const AttnParams& P, int b, int& len) {
  const int n = P.n_nodes ? P.n_nodes[b] : P.N;
  len = P.cache.lens[b];
  const int64_t slots = static_cast<int64_t>(P.cache.max_pages) * P.cache.page_size;
  return n < 1 || n > P.N || len < 0 || len > INT_MAX - 4 * kMaxNodes ||
                 static_cast<int64_t>(len) + n > slots
             ? 0
             : n;
}

// --------------------------------------------------------------- attention

// kPair: more than 128 query rows, two row tiles on the same keys.
template <int DP, bool kPair> struct Shape {
  static constexpr int kTileBytes = kKeys * DP * 2;  // of keys or of values
  static constexpr int kQueryBytes = kRows * DP * 2;
  static constexpr int kStages = 5 * (128 / DP);
  static constexpr int kRowTile = kPair ? 2 * kRows : kRows;
  // shared memory: queries (two tiles: both row tiles, or this and the next item's), stages,
  // then the barriers and what the warps tell one another
  static constexpr int kStageAt = 2 * kQueryBytes;
  static constexpr int kTailAt = kStageAt + kStages * kTileBytes;

  // The order of an item's tiles in the ring, that of the MMAs that read them.
  // One stream: keys a tile ahead of values, K0 K1 V0 K2 V1 .. Kn Vn-1 Vn, so that
  // values do not wait in the ring through their tile's softmax.  Two row tiles:
  // K0 V0 K1 V1 ..
  static __device__ __forceinline__ uint32_t key_job(int i) {
    return kPair ? 2 * i : i ? 2 * i - 1 : 0;
  }
  static __device__ __forceinline__ uint32_t value_job(int i, int tiles) {
    return kPair || i == tiles - 1 ? 2 * i + 1 : 2 * i + 2;
  }
};

// All key tiles t0 .. t1-1 of a row tile that one run has.
struct Item {
  int32_t b, h, row_tile, t0, t1, tiles, len, n;  // t0 < 0: no more items
  int32_t pieces;       // runs that have key tiles of it
  int32_t bad;          // written by the checking warp
  uint8_t parents[kMaxNodes];                          // each below its node, whatever the input

  __device__ __forceinline__ int rows(int group, int row_tile_rows) const {
    return n * group - row_tile * row_tile_rows;
  }
};

template <int kStages> struct Tail {
  uint64_t kv_full[kStages], kv_empty[kStages], q_full[2], q_empty[2], s_full[2], o_full[2];
  uint64_t p_full[2][2];  // by stream and half of the keys
  uint64_t item_full[kItems], item_checked[kItems], item_empty[kItems];
  uint64_t drained;
  uint64_t odd_values[2];  // nodes whose values were not finite, by parity of the item
  unsigned long long total;
  int gave_up;
  uint32_t tmem;
  Item items[kItems];
  float2 stats[2][kRows];
};

// The work units of request b: for each row tile of a key head (an item)
// kItemCost and its 128-key tiles, in this order.
template <int kRowTile>
__device__ __forceinline__ int64_t units_of(const AttnParams& P, int b, int& tiles, int& row_tiles,
                                            int& len, int& n) {
  n = nodes_of(P, b, len);
  tiles = n ? (len + n + kKeys - 1) / kKeys : 0;
  row_tiles = (n * P.group + kRowTile - 1) / kRowTile;
  return n ? static_cast<int64_t>(tiles + kItemCost) * row_tiles * P.cache.heads : 0;
}

// Bits of the 32 columns from `first` (a key's number less len): which of them
// a row sees whose nodes are `visible`.
__device__ __forceinline__ uint32_t seen_of(int first, uint64_t visible) {
  if (first <= -32) return ~0u;
  if (first < 0) return ~(~0u << -first) | static_cast<uint32_t>(visible) << -first;
  return first < 64 ? static_cast<uint32_t>(visible >> first) : 0u;
}

template <class E, int DP, bool kPair>
__global__ void __launch_bounds__(kThreads, 1)
    attention_kernel(const AttnParams P, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map) {
  using S = Shape<DP, kPair>;
  constexpr int kStages = S::kStages;
  // weights in f16 go below 2^-14, where its steps stop shrinking: taken 2^7 larger
  // they reach 2^15 at most (2^kRise more than the maximum's)
  constexpr float kLift = std::is_same<E, F16>::value ? 7.0f : 0.0f;
  extern __shared__ __align__(1024) char smem[];
  Tail<kStages>& s = *reinterpret_cast<Tail<kStages>*>(smem + S::kTailAt);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  const uint32_t base = smem_of(smem);
  const Cache& C = P.cache;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    for (int i = 0; i < kStages; i++) {
      barrier_init(smem_of(&s.kv_full[i]), P.box_rows ? 1 : 32 * kLoadWarps);
      barrier_init(smem_of(&s.kv_empty[i]), 1);
    }
    for (int i = 0; i < 2; i++) {
      barrier_init(smem_of(&s.q_full[i]), 32 * kLoadWarps);
      barrier_init(smem_of(&s.q_empty[i]), 1);
      barrier_init(smem_of(&s.s_full[i]), 1);
      barrier_init(smem_of(&s.p_full[i][0]), 4);
      barrier_init(smem_of(&s.p_full[i][1]), 4);
      barrier_init(smem_of(&s.o_full[i]), 1);
      s.odd_values[i] = 0;
    }
    for (int i = 0; i < kItems; i++) {
      barrier_init(smem_of(&s.item_full[i]), 1);
      barrier_init(smem_of(&s.item_checked[i]), 1);
      barrier_init(smem_of(&s.item_empty[i]), kLoadWarps + 3 + 8);
    }
    barrier_init(smem_of(&s.drained), 2);
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
  int64_t mine = 0;
  for (int b = tid; b < P.B; b += kThreads) {
    int tiles, row_tiles, len, n;
    mine += units_of<S::kRowTile>(P, b, tiles, row_tiles, len, n);
  }
#pragma unroll
  for (int o = 16; o > 0; o /= 2) mine += __shfl_xor_sync(kFullMask, mine, o);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (lane == 0 && mine) atomicAdd(&s.total, static_cast<unsigned long long>(mine));
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

  if (warp >= kLoadWarp && warp < kCheckWarp) {
    // ------------------------------------------------------------- copies
    asm volatile("setmaxnreg.dec.sync.aligned.u32 " SPECV_REGS_LOAD ";");
    // Copies of 16 bytes, so that pages of any size and strides of any kind will
    // do; places without a key (behind the last, past the head) become 0.
    constexpr int kPieces = DP / 8;            // 16-byte pieces of a row
    constexpr int kRowsAtOnce = 32 / kPieces;  // rows of one warp instruction
    const int lw = warp - kLoadWarp, piece = lane % kPieces, sub = lane / kPieces;
    const bool inside = piece * 8 < C.head_dim;
    uint32_t jobs = 0;  // before this item
    uint32_t sent = 0;  // ... and by tensor copies so far
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
      const uint32_t item = items;
      const Item& w = next_item();
      if (__any_sync(kFullMask, over(w))) break;
      const int q_buffer = kPair ? 0 : item & 1;
      const uint32_t q_use = kPair ? item : item / 2;
      const int rows = w.rows(P.group, S::kRowTile);
      if (!__all_sync(kFullMask, barrier_wait(smem_of(&s.q_empty[q_buffer]), (q_use & 1) ^ 1, gave_up)))
        break;
#pragma unroll
      for (int half = 0; half < (kPair ? 2 : 1); half++) {
        const int row = half * kRows + 32 * lw + lane;
        const bool real = row < rows;
        const int at = w.row_tile * S::kRowTile + (real ? row : 0);
        const int node = at / P.group, g = at - node * P.group;
        const int64_t off = w.b * P.q.batch_stride + node * P.q.node_stride +
                            (w.h * P.group + g) * P.q.head_stride;
        tile_copy(base + (kPair ? half : q_buffer) * S::kQueryBytes, P.q.data, real ? off : -1);
      }
      copies_arrive(smem_of(&s.q_full[q_buffer]));
      const int keys = w.len + w.n, t1 = w.t1;
      const int32_t* table = C.page_table + static_cast<int64_t>(w.b) * C.table_stride;
      // Page numbers are read a tile ahead of their use; one out of range (its
      // request is flagged elsewhere) is no page.
      auto page_at = [&](int key) {
        int page = -1;
        if (key < keys) page = table[key / C.page_size];
        return page < C.pages ? page : -1;
      };
      bool going = true;  // the same on every lane
      if (P.box_rows) {
        // Tensor copies: lane l < boxes brings box l % per_half of 64-column half
        // l / per_half.  A page's rows behind the last key come along; the
        // softmax clears their values.
        if (lw == kLoadWarps - 1) {
          const int per_half = kKeys / P.box_rows, boxes = per_half * (DP / 64);
          const int box = lane % per_half, half = lane / per_half;
          const int at = box * P.box_rows;
          auto page_of = [&](int t) {
            return t < t1 && lane < boxes ? page_at(t * kKeys + at) : -1;
          };
          int page = page_of(w.t0), page_next = page_of(w.t0 + 1);
          auto copy = [&](uint32_t job, const CUtensorMap* map, int page, int t) {
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
                          map, half * 64, (t * kKeys + at) % C.page_size, w.h, page, bar);
            return true;
          };
          int page_before = -1;
          for (int t = w.t0; t < t1 && going; t++) {
            const int i = t - w.t0;
            going = copy(S::key_job(i), &k_map, page, t);
            if (going && kPair) going = copy(S::value_job(i, t1 - w.t0), &v_map, page, t);
            else if (going && i > 0) going = copy(S::value_job(i - 1, t1 - w.t0), &v_map, page_before, t - 1);
            page_before = page;
            page = page_next;
            page_next = page_of(t + 2);
          }
          if (going && !kPair)
            going = copy(S::value_job(t1 - 1 - w.t0, t1 - w.t0), &v_map, page_before, t1 - 1);
        }
      } else {
        auto key_of = [&](int t) { return t * kKeys + 32 * lw + lane; };
        auto page_of = [&](int t) { return t < t1 ? page_at(key_of(t)) : -1; };
        int page = page_of(w.t0), page_next = page_of(w.t0 + 1);
        auto copy = [&](uint32_t job, const uint16_t* from, int64_t off) {
          const uint32_t stage = (jobs + job) % kStages, use = (jobs + job) / kStages;
          if (!__all_sync(kFullMask, barrier_wait(smem_of(&s.kv_empty[stage]), (use & 1) ^ 1, gave_up)))
            return false;
          tile_copy(base + S::kStageAt + stage * S::kTileBytes, from, off);
          copies_arrive(smem_of(&s.kv_full[stage]));
          return true;
        };
        int64_t before = -1;
        for (int t = w.t0; t < t1 && going; t++) {
          const int i = t - w.t0;
          const int64_t off = page < 0 ? static_cast<int64_t>(-1)
                                       : page * C.page_stride +
                                             key_of(t) % C.page_size * C.row_stride +
                                             w.h * C.head_stride;
          page = page_next;
          page_next = page_of(t + 2);
          going = copy(S::key_job(i), C.k, off);
          if (going && kPair) going = copy(S::value_job(i, t1 - w.t0), C.v, off);
          else if (going && i > 0) going = copy(S::value_job(i - 1, t1 - w.t0), C.v, before);
          before = off;
        }
        if (going && !kPair) going = copy(S::value_job(t1 - 1 - w.t0, t1 - w.t0), C.v, before);
      }
      if (!going) break;
      jobs += 2 * (t1 - w.t0);
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
  } else if (warp >= kCheckWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 " SPECV_REGS_OTHER ";");
    // --------------------------------------------------------------- MMAs
    constexpr uint32_t kType = std::is_same<E, Bf16>::value ? 1 : 0;
    constexpr uint32_t kIdesc = 1u << 4 | kType << 7 | kType << 10 | (kRows >> 4) << 24;
    constexpr uint32_t kIdescS = kIdesc | (kKeys >> 3) << 17;
    constexpr uint32_t kIdescO = kIdesc | 1u << 16 | (DP >> 3) << 17;
    // Two threads, that neither waits for what the other issues: scores of a tile
    // when its stream's last sum has left S, sums when the weights are there.
    auto stage_at = [&](uint32_t job) { return base + S::kStageAt + job % kStages * S::kTileBytes; };
    auto kv_wait = [&](uint32_t job) {
      const bool there = barrier_wait(smem_of(&s.kv_full[job % kStages]), job / kStages & 1, gave_up);
      // copies of 16 bytes wrote through the generic proxy, the MMA reads through the other
      if (!P.box_rows) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      return there;
    };
    uint32_t jobs = 0;            // copies before this item
    uint32_t issued[2] = {0, 0};  // scores or sums of each stream so far
    if (warp == kScoreWarp && lane == 0) {
      const int steps = (C.head_dim + 15) / 16;
      auto scores = [&](int st, uint32_t q_at, uint32_t k_at) {
        if (issued[st] && !barrier_wait(smem_of(&s.o_full[st]), (issued[st] - 1) & 1, gave_up)) return false;
        tmem_fence_after();
        const uint32_t a = operand_low(q_at, 16), b = operand_low(k_at, 16);
        mma_ss<false>(tS[st], a, b, kIdescS);
#pragma unroll
        for (int k = 1; k < DP / 16; k++) {
          const uint32_t step = ((k / 4) * (kKeys * 128) + (k % 4) * 32) >> 4;  // of both
          if (k < steps) mma_ss<true>(tS[st], a + step, b + step, kIdescS);
        }
        mma_commit(smem_of(&s.s_full[st]));
        issued[st]++;
        return true;
      };
      while (true) {
        const uint32_t item = items;
        const Item& w = next_item();
        if (over(w)) break;
        const int q_buffer = kPair ? 0 : item & 1;
        const uint32_t q_use = kPair ? item : item / 2;
        const bool second = kPair && w.rows(P.group, S::kRowTile) > kRows;
        const int tiles = w.t1 - w.t0;
        done_item();
        bool going = barrier_wait(smem_of(&s.q_full[q_buffer]), q_use & 1, gave_up);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        for (int i = 0; i < tiles && going; i++) {
          const uint32_t job = jobs + S::key_job(i);
          going = kv_wait(job);
          if (kPair) {
            going = going && scores(0, base, stage_at(job));
            if (second) going = going && scores(1, base + S::kQueryBytes, stage_at(job));
          } else {
            going = going && scores(i & 1, base + q_buffer * S::kQueryBytes, stage_at(job));
          }
          if (going) mma_commit(smem_of(&s.kv_empty[job % kStages]));
        }
        if (!going) break;
        jobs += 2 * tiles;
        mma_commit(smem_of(&s.q_empty[q_buffer]));
      }
      // every MMA and every arrival that waits for one must find this CTA's memory
      mma_commit(smem_of(&s.drained));
      barrier_wait_own(smem_of(&s.drained), 0);
    }
    if (warp == kSumWarp && lane == 0) {
      auto sums = [&](int st, uint32_t v_at, bool first) {
        const uint32_t b = operand_low(v_at, kKeys * 128);
#pragma unroll
        for (int half = 0; half < 2; half++) {
          if (!barrier_wait(smem_of(&s.p_full[st][half]), issued[st] & 1, gave_up)) return false;
          tmem_fence_after();
#pragma unroll
          for (int k = half * kKeys / 32; k < (half + 1) * kKeys / 32; k++)
            mma_ts(tO[st], tS[st] + 8 * k, b + (k * 2048 >> 4), kIdescO, k > 0 || !first);
        }
        mma_commit(smem_of(&s.o_full[st]));
        issued[st]++;
        return true;
      };
      while (true) {
        const Item& w = next_item();
        if (over(w)) break;
        const bool second = kPair && w.rows(P.group, S::kRowTile) > kRows;
        const int tiles = w.t1 - w.t0;
        done_item();
        bool going = true;
        for (int i = 0; i < tiles && going; i++) {
          const uint32_t job = jobs + S::value_job(i, tiles);
          going = kv_wait(job);
          if (kPair) {
            going = going && sums(0, stage_at(job), i == 0);
            if (second) going = going && sums(1, stage_at(job), i == 0);
          } else {
            going = going && sums(i & 1, stage_at(job), i < 2);
          }
          if (going) mma_commit(smem_of(&s.kv_empty[job % kStages]));
        }
        if (!going) break;
        jobs += 2 * tiles;
      }
      mma_commit(smem_of(&s.drained));
      barrier_wait_own(smem_of(&s.drained), 0);
    }
    __syncwarp();
    // ------------------------------------------------------------ listing
    if (warp == kListWarp) {
      const Runs runs(P, static_cast<int64_t>(s.total));
      const int run = blockIdx.x;
      int b = 0;           // the request where the search is, ...
      int64_t before = 0;  // ... and the units before it
      bool stop = false, begins = true;
      // every run's, whatever is in it: the join follows what it finds
      if (lane == 0) P.ws.cuts[run] = Cut{0, 0, 0, 0, 0, 0, {0, 0}};
      int64_t u = runs.start(run);
      const int64_t end = runs.start(run + 1);
      while (u < end && !stop) {
        // the request with unit u: 32 requests at a time
        int tiles, row_tiles, len, n;
        int64_t units;
        while (true) {
          units = b + lane < P.B ? units_of<S::kRowTile>(P, b + lane, tiles, row_tiles, len, n) : 0;
          int64_t upto = units;
#pragma unroll
          for (int o = 1; o < 32; o *= 2) {
            const int64_t x = __shfl_up_sync(kFullMask, upto, o);
            if (lane >= o) upto += x;
          }
          const uint32_t past = __ballot_sync(kFullMask, before + upto > u);
          const int from = past ? __ffs(past) - 1 : 31;
          if (past) {
            before += __shfl_sync(kFullMask, upto - units, from);
            b += from;
            tiles = __shfl_sync(kFullMask, tiles, from);
            row_tiles = __shfl_sync(kFullMask, row_tiles, from);
            len = __shfl_sync(kFullMask, len, from);
            n = __shfl_sync(kFullMask, n, from);
            units = __shfl_sync(kFullMask, units, from);
            break;
          }
          before += __shfl_sync(kFullMask, upto, 31);
          b += 32;
          if (b >= P.B) {  // the lengths changed meanwhile
            stop = true;
            break;
          }
        }
        if (stop) break;
        uint8_t up[2];
#pragma unroll
        for (int k = 0; k < 2; k++) {
          const int i = lane + 32 * k;
          int parent = i - 1;
          if (P.parents && i < n) parent = P.parents[static_cast<int64_t>(b) * P.N + i];
          up[k] = static_cast<uint8_t>(parent >= 0 && parent < i ? parent : 0);
        }
        const int span = tiles + kItemCost;
        while (u < end && u < before + units) {
          const int64_t off = u - before;
          const int64_t of = Runs::quotient(off, span);
          const int64_t first = u - (off - of * span) + kItemCost;  // of its tiles' units
          const int h = static_cast<int>(of) / row_tiles;  // below 1024 heads * 512 row tiles
          const int row_tile = static_cast<int>(of) - h * row_tiles;
          const int t0 = static_cast<int>(max(u - first, static_cast<int64_t>(0)));
          const int t1 = static_cast<int>(min(end - first, static_cast<int64_t>(tiles)));
          u = min(end, first + tiles);
          if (t1 <= t0) continue;  // the run ends before the item's first tile
          // runs before and behind with pieces of this item
          int first_run = run, last_run = run;
          if (t0 > 0) first_run = runs.of(first);
          if (t1 < tiles) last_run = runs.of(first + tiles - 1);
          const uint32_t slot = items % kItems;
          barrier_wait(smem_of(&s.item_empty[slot]), (items / kItems & 1) ^ 1, gave_up);
          stop = __any_sync(kFullMask, *gave_up != 0);
          if (stop) break;
          Item& to = s.items[slot];
          to.parents[lane] = up[0];
          to.parents[lane + 32] = up[1];
          if (lane == 0) {
            to.b = b;
            to.h = h;
            to.row_tile = row_tile;
            to.t0 = t0;
            to.t1 = t1;
            to.tiles = tiles;
            to.len = len;
            to.n = n;
            to.pieces = last_run - first_run + 1;
            if (begins && t0 > 0 && first_run == run - 1)
              P.ws.cuts[run] = Cut{b, h, row_tile, n, last_run - first_run + 1, 0, {0, 0}};
          }
          __syncwarp();
          if (lane == 0) barrier_arrive(smem_of(&s.item_full[slot]));
          items++;
          begins = false;
        }
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
      const int64_t slots = static_cast<int64_t>(C.max_pages) * C.page_size;
      auto check = [&](int b, int& n) {
        Tree t = read_tree(P.parents, P.n_nodes, C.lens, b, P.N, slots, lane);
        if (!t.bad && __any_sync(kFullMask, bad_pages(C, b, 0, t.len + t.n, lane, 32)))
          t.bad |= SPECV_DEV_BAD_CACHE;
        n = t.n;
        return t.bad;
      };
      int next = blockIdx.x, last = -1, last_bad = 0, n;
      auto report = [&]() {
        const unsigned bad = check(next, n);
        if (lane == 0) P.status[next] = static_cast<int32_t>(bad);
        int len;
        if (bad && nodes_of(P, next, len) == 0) {  // no item has its rows
          n = n ? n : P.N;
          const int words = C.head_dim / 8;
          for (int e = lane; e < n * P.q_heads * words; e += 32) {
            const int i = e / (P.q_heads * words), h = e / words % P.q_heads, d = e % words * 8;
            *reinterpret_cast<uint4*>(P.out.data + next * P.out.batch_stride +
                                      i * P.out.node_stride + h * P.out.head_stride + d) =
                make_uint4(0, 0, 0, 0);
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
        if (w.b != last) last_bad = static_cast<int>(check(w.b, n));
        last = w.b;
        if (lane == 0) w.bad = last_bad;
        __syncwarp();
        if (lane == 0) barrier_arrive(smem_of(&s.item_checked[slot]));
        done_item();
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 " SPECV_REGS_SOFTMAX ";");
    const int st = warp / 4, quarter = warp % 4;
    const int row = quarter * 32 + lane;  // of the stream's tile
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const float c = P.scale_log2;
    uint32_t jobs = 0, scored = 0;  // scored: tiles of this stream so far
    while (true) {
      const uint32_t item = items;
      const Item& given = next_item();
      if (any_of_softmax(over(given))) break;  // all leave together
      const struct {
        int b, h, row_tile, t0, t1, tiles, len, n;
      } w = {given.b, given.h, given.row_tile, given.t0, given.t1, given.tiles, given.len, given.n};
      const int rows = given.rows(P.group, S::kRowTile);
      const int first_row = kPair ? st * kRows : 0;
      const bool second = !kPair || rows > kRows;
      const bool working = first_row + quarter * 32 < rows;  // this warp has rows
      const int at = w.row_tile * S::kRowTile + min(first_row + row, rows - 1);
      const int node = at / P.group, g = at - node * P.group;
      uint64_t visible = 1;  // nodes that this row sees: its own and those above it
      if (w.t1 * kKeys > w.len)
        for (int i = node; i > 0; i = given.parents[i]) visible |= 1ull << i;
      const int keys = w.len + w.n;
      uint64_t* odd = &s.odd_values[item & 1];
      int taken[2] = {0, 0};  // tiles of this item that each stream took
      float m = -INFINITY, l = 0.0f;  // m: the maximum that O and l were taken with, times c

      for (int t = w.t0; t < w.t1; t++) {
        if (kPair) {
          taken[0]++;
          if (second) taken[1]++;
          if (st == 1 && !second) continue;
        } else {
          // by the item's own count, so that a row's sums do not depend on what ran before
          taken[(t - w.t0) & 1]++;
          if (((t - w.t0) & 1) != st) continue;
        }
        if (!__all_sync(kFullMask, barrier_wait(smem_of(&s.s_full[st]), scored & 1, gave_up))) break;
        const bool mixed = (t + 1) * kKeys > w.len;  // holds keys that not every row sees
        if (mixed && (!kPair || st == 0)) {
          // (Only now that the scores are there: a wait tells phases apart by their parity,
          // so the copy before this one in the same stage must be known to have landed.)
          // A value that is not finite would pass through a weight of 0 into rows that do
          // not see its node: it becomes 0 here and comes back, at the end, for those that do.
          const uint32_t job = jobs + S::value_job(t - w.t0, w.t1 - w.t0), stage = job % kStages;
          if (!__all_sync(kFullMask, barrier_wait(smem_of(&s.kv_full[stage]), job / kStages & 1, gave_up)))
            break;
          char* v = smem + S::kStageAt + stage * S::kTileBytes;
          const int from = max(w.len - t * kKeys, 0), to = min(keys - t * kKeys, kKeys);
          // (and a tensor copy's rows behind the last key hold whatever the page has)
          const int stale = P.box_rows ? kKeys - to : 0;
          constexpr uint32_t kExp = std::is_same<E, Bf16>::value ? 0x7f80u : 0x7c00u;
          bool changed = false;
          for (int e = (quarter * 32 + lane); e < (to - from) * (DP / 8); e += 128) {
            const int r = from + e / (DP / 8), p = e % (DP / 8);
            uint4* place = reinterpret_cast<uint4*>(v + (p / 8) * (kKeys * 128) + r * 128 + (p % 8) * 16);
            uint4 x = *place;
            uint32_t* words = &x.x;
            bool found = false;
#pragma unroll
            for (int i = 0; i < 4; i++) {
              if ((words[i] & kExp) == kExp) words[i] &= 0xffff0000u, found = true;
              if ((words[i] >> 16 & kExp) == kExp) words[i] &= 0xffffu, found = true;
            }
            if (found) {
              *place = x;
              atomicOr(reinterpret_cast<unsigned long long*>(odd),
                       1ull << (t * kKeys + r - w.len));
              changed = true;
            }
          }
          for (int e = quarter * 32 + lane; e < stale * (DP / 8); e += 128) {
            const int r = to + e / (DP / 8), p = e % (DP / 8);
            *reinterpret_cast<uint4*>(v + (p / 8) * (kKeys * 128) + r * 128 + (p % 8) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          if (changed || stale) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        __syncwarp();
        tmem_fence_after();
        const bool first = taken[st] == 1;
        if (working) {
          uint32_t x[kKeys];
          tmem_load128(tS[st] + lanes, x);
          if (mixed) {
#pragma unroll
            for (int k = 0; k < kKeys; k += 32) {
              const uint32_t seen = seen_of(t * kKeys + k - w.len, visible);
#pragma unroll
              for (int e = 0; e < 32; e++)
                if (!(seen >> e & 1)) x[k + e] = 0xff800000u;  // -inf
            }
          }
          float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < kKeys; e += 8)
#pragma unroll
            for (int k = 0; k < 4; k++)
              tops[k] = fmaxf(fmaxf(tops[k], __uint_as_float(x[e + 2 * k])),
                              __uint_as_float(x[e + 2 * k + 1]));
          const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * c;
          const bool rise = first || top > m + kRise;
          float by = 1.0f;
          if (rise) {
            const float higher = fmaxf(m, top);
            by = higher == -INFINITY ? 1.0f : exp2_of(m - higher);
            m = higher;
          }
          if (!first && __any_sync(kFullMask, rise)) {
            // the last update of O must be done
            if (!__all_sync(kFullMask, barrier_wait(smem_of(&s.o_full[st]), (scored - 1) & 1, gave_up)))
              break;
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
          const float shift = kLift - (m == -INFINITY ? 0.0f : m);
          const uint64_t c2 = pair_of(__float_as_uint(c), __float_as_uint(c));
          const uint64_t shift2 = pair_of(__float_as_uint(shift), __float_as_uint(shift));
          uint64_t sums[2] = {0, 0};
#pragma unroll
          for (int k = 0; k < kKeys; k += 32) {
            uint32_t p[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 y = halves_of(fma2(pair_of(x[k + e], x[k + e + 1]), c2, shift2));
              const float a = exp2_of(y.x), b = exp2_of(y.y);
              sums[e / 2 % 2] =
                  add2(sums[e / 2 % 2], pair_of(__float_as_uint(a), __float_as_uint(b)));
              // the weights' one rounding, to the type of the values they meet: the MMA takes
              // both operands in one 16-bit type.  (The sum has them as they are.  Against 64 bits
              // the output is off by 2.2e-3 of its size in bf16, 2.9e-4 in f16; by 1.6e-3 and
              // 2.1e-4 with weights in 32 bits, the output's own rounding.)
              p[e / 2] = E::pack(a, b);
            }
            tmem_store16(tS[st] + lanes + k / 2, p);  // over scores of this row, all read
            if (k == kKeys / 2 - 32) {  // half of the keys can be summed up
              tmem_store_wait();
              tmem_fence_before();
              __syncwarp();
              if (lane == 0) barrier_arrive(smem_of(&s.p_full[st][0]));
            }
          }
          const float2 sum = halves_of(add2(sums[0], sums[1]));
          l += sum.x + sum.y;
          tmem_store_wait();
        } else if (lane == 0) {
          barrier_arrive(smem_of(&s.p_full[st][0]));
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) barrier_arrive(smem_of(&s.p_full[st][1]));
        scored++;
      }

      jobs += 2 * (w.t1 - w.t0);

      // The item's end: this stream's last sum, and by the barrier the other's too.
      if (taken[st]) barrier_wait(smem_of(&s.o_full[st]), (scored - 1) & 1, gave_up);
      s.stats[st][row] = make_float2(m, l);
      tmem_fence_before();
      asm volatile("bar.sync 1, 256;" ::: "memory");
      tmem_fence_after();
      const uint64_t odd_rows = *odd & visible;
      const float2 other = s.stats[st ^ 1][row];
      if (tid == 0) s.odd_values[(item & 1) ^ 1] = 0;
      barrier_wait(smem_of(&s.item_checked[items % kItems]), items / kItems & 1, gave_up);
      const bool bad = __any_sync(kFullMask, given.bad != 0 || *gave_up);  // unchecked is bad
      // Only a checked request's pages are followed.  (Of a flagged one a box may not have
      // been copied, and what its place in the ring held before may look like such values.)
      const uint64_t fix = bad ? 0 : odd_rows;
      const int pieces = given.pieces;
      __syncwarp();
      done_item();
      // kPair: this stream's rows, all columns; else half of the columns of both streams' sum
      const int my_rows = rows - first_row;
      if (quarter * 32 < my_rows && !(bad && w.t0 > 0)) {
        float weight[2] = {1.0f, 1.0f};
        if (!kPair) {
          const float m_of[2] = {st ? other.x : m, st ? m : other.x};
          const float l_of[2] = {st ? other.y : l, st ? l : other.y};
          m = fmaxf(m_of[0], m_of[1]);
          l = 0.0f;
#pragma unroll
          for (int k = 0; k < 2; k++) {
            weight[k] = !taken[k] ? 0.0f : m_of[k] == m ? 1.0f : exp2_of(m_of[k] - m);
            l += weight[k] * l_of[k];
          }
        }
        const bool whole = pieces == 1 || bad;  // of a flagged request the first piece clears the rows
        const float inv = 1.0f / l;
        const bool mine = row < my_rows;
        uint16_t* out = P.out.data + w.b * P.out.batch_stride + node * P.out.node_stride +
                        (w.h * P.group + g) * P.out.head_stride;
        const int64_t slot = 2 * static_cast<int>(blockIdx.x) + (w.t0 == 0);
        float4* part = P.ws.parts + slot * (DP / 4) * P.part_rows + first_row + row;
        constexpr int kCols = kPair ? DP : DP / 2;
        const int col0 = kPair ? 0 : st * kCols;
#pragma unroll 1
        for (int k = 0; k < kCols; k += 32) {
          float o[32];
          uint32_t x[32];
          if (kPair) {
            tmem_load32(tO[st] + lanes + k, x);
#pragma unroll
            for (int e = 0; e < 32; e++) o[e] = __uint_as_float(x[e]);
          } else {
#pragma unroll
            for (int e = 0; e < 32; e++) o[e] = 0.0f;
#pragma unroll
            for (int i = 0; i < 2; i++)
              if (taken[i]) {
                tmem_load32(tO[i] + lanes + col0 + k, x);
#pragma unroll
                for (int e = 0; e < 32; e++) o[e] = fmaf(__uint_as_float(x[e]), weight[i], o[e]);
              }
          }
          if (mine) {
            for (uint64_t left = fix; left; left &= left - 1) {
              const uint16_t* v = C.v + C.slot(w.b, w.len + __ffsll(left) - 1) + w.h * C.head_stride;
              constexpr uint32_t kExp = std::is_same<E, Bf16>::value ? 0x7f80u : 0x7c00u;
#pragma unroll
              for (int e = 0; e < 32; e++) {
                const int d = col0 + k + e;
                if (d >= C.head_dim) continue;
                const uint32_t bits = v[d];
                if ((bits & kExp) == kExp) o[e] += E::unpack(bits).x;
              }
            }
          }
          if (mine && whole) {
            if (bad)
#pragma unroll
              for (int e = 0; e < 32; e++) o[e] = 0.0f;
            const float by = bad ? 0.0f : inv;
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              const int d = col0 + k + e;
              if (d < C.head_dim)
                *reinterpret_cast<uint4*>(out + d) =
                    make_uint4(E::pack(o[e] * by, o[e + 1] * by),
                               E::pack(o[e + 2] * by, o[e + 3] * by),
                               E::pack(o[e + 4] * by, o[e + 5] * by),
                               E::pack(o[e + 6] * by, o[e + 7] * by));
            }
          } else if (mine) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              part[(col0 + k + e) / 4 * P.part_rows] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
          __syncwarp();
        }
        if (!whole && mine && (kPair || st == 0)) 
          P.ws.stats[slot * P.part_rows + first_row + row] = make_float2(m, l);
      }
      tmem_fence_before();
      asm volatile("bar.sync 1, 256;" ::: "memory");
      tmem_fence_after();
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
// A block to a run's cut, or to 16 of its rows; that of a run that gave up flags the
// whole call (whose statuses are all written by now).  A warp takes eight rows and kJoinPieces
// pieces at a time, all of their loads in flight; with kShares > 1 the warps share
// out the pieces.  A lane has one row and every fourth four columns
// of it.  The code is short on purpose: it runs once, and fetching it was most
// of the time of an unrolled form.
constexpr int kJoinRows = 8;

template <class E, int DP, int kRowTile, int kJoinWarps, int kRowGroups>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const AttnParams P) {
  constexpr int kShares = kJoinWarps / kRowGroups;
  constexpr int kJoinPieces = kShares > 1 ? 4 : 2;
  constexpr int kQuads = DP / 16;  // of a lane
  __shared__ float4 s_o[kShares > 1 ? kJoinWarps : 1][kQuads][32];
  __shared__ float2 s_ml[kJoinWarps][kJoinRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int group = warp % kRowGroups, share = warp / kRowGroups;
  const int run = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Cut cut = P.ws.cuts[run];
  if (cut.gave_up && blockIdx.y == 0)
    for (int b = threadIdx.x; b < P.B; b += kJoinWarps * 32) atomicOr(P.status + b, SPECV_DEV_TIMEOUT);
  // (A call that gave up may leave records of another: they are not followed out of bounds.)
  if (cut.pieces < 2 || cut.pieces > P.ctas - run + 1 || cut.b < 0 || cut.b >= P.B ||
      cut.h < 0 || cut.h >= P.cache.heads || cut.n < 1 || cut.n > P.N || cut.row_tile < 0 ||
      cut.row_tile * kRowTile >= cut.n * P.group)
    return;
  const int rows = min(kRowTile, cut.n * P.group - cut.row_tile * kRowTile);
  const int flagged = P.status[cut.b];  // its first piece has cleared the rows
  const int row = lane % kJoinRows, quad = lane / kJoinRows;
  const int first = blockIdx.y * (kRowGroups * kJoinRows);
#pragma unroll 1
  for (int row0 = first + group * kJoinRows;
       kShares > 1 ? first < rows : row0 < rows; row0 += kRowGroups * kJoinRows) {
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
    for (int i0 = share * kJoinPieces; i0 < cut.pieces; i0 += kShares * kJoinPieces) {
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
    if (kShares > 1) {
      // the warps' shares, in their order
      if (quad == 0) s_ml[warp][row] = make_float2(m, l);
#pragma unroll
      for (int j = 0; j < kQuads; j++) s_o[warp][j][lane] = o[j];
      __syncthreads();
      if (share) return;
#pragma unroll 1
      for (int w = 1; w < kShares; w++) {
        const float2 ml = s_ml[warp + w * kRowGroups][row];
        const float top = fmaxf(m, ml.x);
        const float old = m == top ? 1.0f : exp2_of(m - top);
        const float by = ml.x == top ? 1.0f : exp2_of(ml.x - top);
        m = top;
        l = fmaf(by, ml.y, l * old);
        add(old, by, &s_o[warp + w * kRowGroups][0][lane], 32);
      }
    }
    // (shared pieces: this is the only round, whatever rows there are)
    if (row0 + row >= rows || flagged) {
      if (kShares > 1) return;
      continue;
    }
    const float inv = 1.0f / l;
    const int flat = cut.row_tile * kRowTile + row0 + row, node = flat / P.group, g = flat - node * P.group;
    uint16_t* out = P.out.data + cut.b * P.out.batch_stride + node * P.out.node_stride +
                    (cut.h * P.group + g) * P.out.head_stride;
#pragma unroll
    for (int j = 0; j < kQuads; j++) {
      const int d = 4 * (quad + 4 * j);
      if (d < P.cache.head_dim)
        *reinterpret_cast<uint2*>(out + d) = make_uint2(E::pack(o[j].x * inv, o[j].y * inv),
                                                        E::pack(o[j].z * inv, o[j].w * inv));
    }
    if (kShares > 1) return;
  }
}

// ------------------------------------------------------------------- host

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// The shape of the work that B, N and the heads give, whatever the lengths are.
struct Plan {
  bool pair;
  int dim, row_tile, part_rows;
  size_t stats, parts, total;  // offsets in the workspace; before them the cuts

  Plan(int N, int group, int head_dim) {
    const int rows = N * group;
    pair = rows > kRows;
    dim = head_dim <= 64 ? 64 : 128;
    row_tile = pair ? 2 * kRows : kRows;
    part_rows = (rows < row_tile ? rows : row_tile) + 7 & ~7;
    stats = align256(kMaxCtas * sizeof(Cut));
    parts = stats + align256(2 * kMaxCtas * part_rows * sizeof(float2));
    total = parts + align256(2 * kMaxCtas * part_rows * dim * sizeof(float));
  }
};

template <class E, int DP, bool kPair>
cudaError_t run(const AttnParams& P, const CUtensorMap& k_map, const CUtensorMap& v_map,
                cudaStream_t stream) {
  using S = Shape<DP, kPair>;
  constexpr int kSmem = S::kTailAt + static_cast<int>(sizeof(Tail<S::kStages>));
  static_assert(kSmem <= 232448, "one CTA's shared memory");
  cudaError_t e = cudaFuncSetAttribute(attention_kernel<E, DP, kPair>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  attention_kernel<E, DP, kPair><<<P.ctas, kThreads, kSmem, stream>>>(P, k_map, v_map);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  // Few rows, or few items (then pieces are many): blocks of 16 rows whose warps share
  // out the pieces (64 nodes over 30,000 keys of one head 44 us, 205 with the last form;
  // 24 items 45 us and 48, 64 items 58 and 47, 64-node trees 388 and 359).
  const int64_t items = static_cast<int64_t>(P.B) * P.cache.heads *
                        ((P.N * P.group + S::kRowTile - 1) / S::kRowTile);
  const bool shared = P.part_rows <= 16 || items < kSms / 4;
  cfg.gridDim = dim3(P.ctas, shared ? (P.part_rows + 15) / 16 : 1);
  cfg.blockDim = dim3(shared || P.part_rows <= 32 ? 256 : 512);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (shared) return cudaLaunchKernelEx(&cfg, join_kernel<E, DP, S::kRowTile, 8, 2>, P);
  if (P.part_rows <= 32) return cudaLaunchKernelEx(&cfg, join_kernel<E, DP, S::kRowTile, 8, 4>, P);
  return cudaLaunchKernelEx(&cfg, join_kernel<E, DP, S::kRowTile, 16, 16>, P);
}

template <class E>
cudaError_t run_any(const AttnParams& P, const Plan& plan, const CUtensorMap& k, const CUtensorMap& v,
                    cudaStream_t stream) {
  if (plan.dim == 64) return plan.pair ? run<E, 64, true>(P, k, v, stream) : run<E, 64, false>(P, k, v, stream);
  return plan.pair ? run<E, 128, true>(P, k, v, stream) : run<E, 128, false>(P, k, v, stream);
}

}  // namespace

extern "C" {

size_t specv_attention_workspace_bytes(int B, int N, int q_heads, int kv_heads, int head_dim) {
  if (B < 1 || B > SPECV_MAX_BATCH || N < 1 || N > SPECV_MAX_NODES || kv_heads < 1 ||
      q_heads < kv_heads || q_heads > 1024 || q_heads % kv_heads != 0 || head_dim < 8 ||
      head_dim > SPECV_MAX_HEAD_DIM || head_dim % 8 != 0)
    return 0;
  return Plan(N, q_heads / kv_heads, head_dim).total;
}

specv_status spec_tree_attention(const specv_cache* cache, const specv_rows* q,
                                 const int32_t* parents, const int32_t* n_nodes, int B, int N,
                                 int q_heads, float scale, const specv_rows* out, int32_t* status,
                                 void* workspace, size_t workspace_bytes, specv_stream_t stream) {
  const specv_status s = check_cache(cache, B, N);
  if (s != SPECV_OK) return s;
  if (!rows_ok(q) || !rows_ok(out) || !status || !workspace || cache->layers != 1 || q_heads < 1 ||
      q_heads % cache->heads != 0 || !(scale > 0.0f) || scale > 2e38f)
    return SPECV_ERR_INVALID_ARG;
  if (!aligned_to(parents, 4) || !aligned_to(n_nodes, 4) || !aligned_to(status, 4) ||
      !aligned_to(workspace, 256))
    return SPECV_ERR_INVALID_ARG;
  if (q_heads > 1024) return SPECV_ERR_UNSUPPORTED;
  const int group = q_heads / cache->heads;
  const Plan plan(N, group, cache->head_dim);
  if (workspace_bytes < plan.total) return SPECV_ERR_WORKSPACE;
  int device = 0, ctas = 0;
  if (cudaGetDevice(&device) != cudaSuccess ||
      cudaDeviceGetAttribute(&ctas, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
    return SPECV_ERR_CUDA;
  if (ctas > kMaxCtas) ctas = kMaxCtas;
  char* base = static_cast<char*>(workspace);
  const Workspace ws{reinterpret_cast<Cut*>(base),
                     reinterpret_cast<float2*>(base + plan.stats),
                     reinterpret_cast<float4*>(base + plan.parts)};
  const int page = cache->page_size;
  // Tensor copies, the largest that fit pages and tiles alike, from 32 rows on, of pairs
  // of row tiles from 16; smaller ones take longer than pieces of 16 bytes (eight chains:
  // of 32 rows 135 us and 139 in pieces, of 16 157 and 145, of 8 238 and 150; 64-node
  // trees: 360 and 404, 388 and 405, 522 and 404).
  const int fit = page & -page;
  int box_rows = fit < (plan.pair ? 16 : 32) ? 0 : fit < kKeys ? fit : kKeys;
  CUtensorMap k_map = {}, v_map = {};
  if (box_rows && (!tensor_map(&k_map, cache, cache->k, box_rows) ||
                   !tensor_map(&v_map, cache, cache->v, box_rows)))
    box_rows = 0;
  const AttnParams P{to_cache(cache),
                     to_rows(q),
                     to_rows(out),
                     ws,
                     parents,
                     n_nodes,
                     status,
                     B,
                     N,
                     q_heads,
                     group,
                     ctas,
                     plan.part_rows,
                     box_rows,
                     scale * 1.4426950408889634f};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->dtype == SPECV_BF16 ? run_any<Bf16>(P, plan, k_map, v_map, st)
                                                   : run_any<F16>(P, plan, k_map, v_map, st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return SPECV_ERR_CUDA;
  }
  return SPECV_OK;
}

}  // extern "C"
