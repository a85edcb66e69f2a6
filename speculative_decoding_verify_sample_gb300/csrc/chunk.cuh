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
// warps: an item of more than 128 rows is a pair of row tiles on the same keys,
// one of fewer takes its key tiles in turn and is joined at the end.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "cache.cuh"
#include "tensor.cuh"

namespace specv_chunk {

using namespace specv_cache_ops;
using namespace specv_tensor;

constexpr int kKeys = 128;     // keys of a tile
constexpr int kRows = 128;     // query rows of a stream
constexpr int kRowTile = 256;  // and of an item
static_assert(kKeys == kRows, "tiles of queries, keys and values are laid out alike");
constexpr int kMaxCtas = kSms;
constexpr int kMaxRequests = SPECV_MAX_CHUNK_REQUESTS;
constexpr int kLoadWarps = 4;
constexpr int kLoadWarp = 8;  // the first of them; the last makes the tensor copies
constexpr int kCheckWarp = 12;
constexpr int kScoreWarp = 13;  // issues S = Q K^T
constexpr int kSumWarp = 14;    // issues O += P V
constexpr int kListWarp = 15;
constexpr int kThreads = 512;
constexpr int kItems = 4;  // items listed ahead
// What an item takes besides its key tiles, in their time: its end, and the next
// one's first scores.
constexpr int kItemCost = 3;
// Registers a thread of each warpgroup: 2 * 192 + 72 + 56 = 512 = 4 * 128, what
// the block is launched with.  The softmax keeps a row of scores in them.
#define SPECV_CHUNK_REGS_SOFTMAX "192"
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
  float cap_log2, cap_turn;           // cap log2 e and 2 scale log2 e / cap; 0: no cap
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
__device__ __forceinline__ int lowest(const Params& P, int pos) {
  return P.window > pos ? 0 : pos - P.window + 1;
}

// The 128-key tiles of an item: numbers 0 .. tiles-1, tile i being keys from
// 128 i on, or 128 (i + skip) from number `gap` on.
struct Span {
  int rows, pos0, pos1, tiles, gap, skip;
};

__device__ __forceinline__ Span span_of(const Params& P, const Request& r, int row_tile) {
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

// An item's units of work: kItemCost and its tiles, a pair's twice.
__device__ __forceinline__ int units_of(const Span& s) {
  return (s.tiles + kItemCost) * (s.rows > kRows ? 2 : 1);
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

  // The order of an item's tiles in the ring, that of the MMAs that read them.
  // In turn: keys a tile ahead of values, K0 K1 V0 K2 V1 .. Kn Vn-1 Vn, so that
  // values do not wait in the ring through their tile's softmax.  A pair:
  // K0 V0 K1 V1 ..
  static __device__ __forceinline__ uint32_t key_job(bool pair, int i) {
    return pair ? 2 * i : i ? 2 * i - 1 : 0;
  }
  static __device__ __forceinline__ uint32_t value_job(bool pair, int i, int tiles) {
    return pair || i == tiles - 1 ? 2 * i + 1 : 2 * i + 2;
  }
};

// Tiles number t0 .. t1-1 of an item that one run has.
struct Item {
  int32_t b, h, row_tile, t0, t1, gap, skip, rows;  // t0 < 0: no more items
  int32_t first, n, len, prefix;
  int32_t pieces;  // runs that have tiles of it
  int32_t begins;  // this is its first piece
  int32_t bad;     // written by the checking warp

  __device__ __forceinline__ int tile(int t) const { return t < gap ? t : t + skip; }
};

// Keys that some rows of an item see and others do not: behind the first row's
// own (up to 255), and below the last row's window (as many).  A bit each.
constexpr int kEdge = 8;

template <int kStages> struct Tail {
  uint64_t kv_full[kStages], kv_empty[kStages], q_full[2], q_empty[2], s_full[2], o_full[2];
  uint64_t p_full[2][2];  // by stream and half of the keys
  uint64_t item_full[kItems], item_checked[kItems], item_empty[kItems];
  uint64_t drained;
  uint32_t odd[2][2 * kEdge];  // edge keys whose values were not finite, by parity of the item
  unsigned long long total;
  int gave_up;
  uint32_t tmem;
  Item items[kItems];
  float2 stats[2][kRows];
};

template <class E, int DP, bool kMod>
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
      barrier_init(smem_of(&s.kv_empty[i]), 1);
    }
    for (int i = 0; i < 2; i++) {
      barrier_init(smem_of(&s.q_full[i]), 32 * kLoadWarps);
      barrier_init(smem_of(&s.q_empty[i]), 1);
      barrier_init(smem_of(&s.s_full[i]), 1);
      barrier_init(smem_of(&s.p_full[i][0]), 4);
      barrier_init(smem_of(&s.p_full[i][1]), 4);
      barrier_init(smem_of(&s.o_full[i]), 1);
      for (int k = 0; k < 2 * kEdge; k++) s.odd[i][k] = 0;
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

  if (warp >= kLoadWarp && warp < kCheckWarp) {
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
      const int at = w.row_tile * kRowTile;
      const int low = lowest(P, w.len + at / P.group);
      const int high = max(w.len + (at + w.rows - 1) / P.group + 1, w.prefix);
      const int t0 = w.t0, t1 = w.t1, tiles = t1 - t0;
      const int32_t* table = C.page_table + static_cast<int64_t>(w.b) * C.table_stride;
      // Page numbers are read a tile ahead of their use; one out of range (its
      // request is flagged elsewhere) is no page.  Of keys key .. key+count-1, of one page:
      auto page_at = [&](int key, int count) {
        int page = -1;
        if (key < high && (key < w.prefix || key + count > low)) page = table[key / C.page_size];
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
          auto page_of = [&](int t) {
            return t < t1 && lane < boxes ? page_at(w.tile(t) * kKeys + at, P.box_rows) : -1;
          };
          int page = page_of(t0), page_next = page_of(t0 + 1);
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
                          map, half * 64, (w.tile(t) * kKeys + at) % C.page_size, w.h, page, bar);
            return true;
          };
          int page_before = -1;
          for (int t = t0; t < t1 && going; t++) {
            const int i = t - t0;
            going = copy(S::key_job(pair, i), &k_map, page, t);
            if (going && pair) going = copy(S::value_job(pair, i, tiles), &v_map, page, t);
            else if (going && i > 0) going = copy(S::value_job(pair, i - 1, tiles), &v_map, page_before, t - 1);
            page_before = page;
            page = page_next;
            page_next = page_of(t + 2);
          }
          if (going && !pair)
            going = copy(S::value_job(pair, tiles - 1, tiles), &v_map, page_before, t1 - 1);
        }
      } else {
        auto key_of = [&](int t) { return w.tile(t) * kKeys + 32 * lw + lane; };
        auto page_of = [&](int t) { return t < t1 ? page_at(key_of(t), 1) : -1; };
        int page = page_of(t0), page_next = page_of(t0 + 1);
        auto copy = [&](uint32_t job, const uint16_t* from, int64_t off) {
          const uint32_t stage = (jobs + job) % kStages, use = (jobs + job) / kStages;
          if (!__all_sync(kFullMask, barrier_wait(smem_of(&s.kv_empty[stage]), (use & 1) ^ 1, gave_up)))
            return false;
          tile_copy(base + S::kStageAt + stage * S::kTileBytes, from, off);
          copies_arrive(smem_of(&s.kv_full[stage]));
          return true;
        };
        int64_t before = -1;
        for (int t = t0; t < t1 && going; t++) {
          const int i = t - t0;
          const int64_t off = page < 0 ? static_cast<int64_t>(-1)
                                       : page * C.page_stride +
                                             key_of(t) % C.page_size * C.row_stride +
                                             w.h * C.head_stride;
          page = page_next;
          page_next = page_of(t + 2);
          going = copy(S::key_job(pair, i), C.k, off);
          if (going && pair) going = copy(S::value_job(pair, i, tiles), C.v, off);
          else if (going && i > 0) going = copy(S::value_job(pair, i - 1, tiles), C.v, before);
          before = off;
        }
        if (going && !pair) going = copy(S::value_job(pair, tiles - 1, tiles), C.v, before);
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
  } else if (warp >= kCheckWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 " SPECV_CHUNK_REGS_OTHER ";");
    // --------------------------------------------------------------- MMAs
    constexpr uint32_t kType = std::is_same<E, Bf16>::value ? 1 : 0;
    constexpr uint32_t kIdesc = 1u << 4 | kType << 7 | kType << 10 | (kRows >> 4) << 24;
    constexpr uint32_t kIdescS = kIdesc | (kKeys >> 3) << 17;
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
    const int steps = (C.head_dim + 15) / 16;
    if (warp == kScoreWarp && lane == 0) {
      uint32_t queries = 0;
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
        const Item& w = next_item();
        if (over(w)) break;
        const bool pair = w.rows > kRows;
        const int tiles = w.t1 - w.t0;
        done_item();
        bool going = true;
        uint32_t q_at[2];
        for (int half = 0; half < (pair ? 2 : 1) && going; half++) {
          const uint32_t buffer = (queries + half) & 1;
          going = barrier_wait(smem_of(&s.q_full[buffer]), (queries + half) / 2 & 1, gave_up);
          q_at[half] = base + buffer * S::kQueryBytes;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        for (int i = 0; i < tiles && going; i++) {
          const uint32_t job = jobs + S::key_job(pair, i);
          going = kv_wait(job);
          if (pair) {
            going = going && scores(0, q_at[0], stage_at(job));
            going = going && scores(1, q_at[1], stage_at(job));
          } else {
            going = going && scores(i & 1, q_at[0], stage_at(job));
          }
          if (going) mma_commit(smem_of(&s.kv_empty[job % kStages]));
        }
        if (!going) break;
        jobs += 2 * tiles;
        for (int half = 0; half < (pair ? 2 : 1); half++, queries++)
          mma_commit(smem_of(&s.q_empty[queries & 1]));
      }
      // every MMA and every arrival that waits for one must find this CTA's memory
      mma_commit(smem_of(&s.drained));
      barrier_wait_own(smem_of(&s.drained), 0);
    }
    if (warp == kSumWarp && lane == 0) {
      const uint32_t idesc = kIdesc | 1u << 16 | static_cast<uint32_t>(2 * steps) << 17;
      auto sums = [&](int st, uint32_t v_at, bool first) {
        const uint32_t b = operand_low(v_at, kKeys * 128);
#pragma unroll
        for (int half = 0; half < 2; half++) {
          if (!barrier_wait(smem_of(&s.p_full[st][half]), issued[st] & 1, gave_up)) return false;
          tmem_fence_after();
#pragma unroll
          for (int k = half * kKeys / 32; k < (half + 1) * kKeys / 32; k++)
            mma_ts(tO[st], tS[st] + 8 * k, b + (k * 2048 >> 4), idesc, k > 0 || !first);
        }
        mma_commit(smem_of(&s.o_full[st]));
        issued[st]++;
        return true;
      };
      while (true) {
        const Item& w = next_item();
        if (over(w)) break;
        const bool pair = w.rows > kRows;
        const int tiles = w.t1 - w.t0;
        done_item();
        bool going = true;
        for (int i = 0; i < tiles && going; i++) {
          const uint32_t job = jobs + S::value_job(pair, i, tiles);
          going = kv_wait(job);
          if (pair) {
            going = going && sums(0, stage_at(job), i == 0);
            going = going && sums(1, stage_at(job), i == 0);
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
          const int64_t first = before + h * head + passed + weight * kItemCost;
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
                                 r.len, r.prefix, pieces, t0 == 0, 0};
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
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 " SPECV_CHUNK_REGS_SOFTMAX ";");
    const int st = warp / 4, quarter = warp % 4;
    const int row = quarter * 32 + lane;  // of the stream's tile
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const float c = P.scale_log2;
    uint32_t jobs = 0, scored = 0;  // scored: tiles of this stream so far
    while (true) {
      const uint32_t item = items;
      const Item& given = next_item();
      if (any_of_softmax(over(given))) break;  // all leave together
      const Item w = given;
      const bool pair = w.rows > kRows;
      const int first_row = pair ? st * kRows : 0;
      const bool working = first_row + quarter * 32 < w.rows;  // this warp has rows
      const int item_row = w.row_tile * kRowTile;
      const int at = item_row + min(first_row + row, w.rows - 1);
      const int token = at / P.group, g = at - token * P.group;
      // slots that this row sees: below the prefix, and low .. pos
      const int pos = w.len + token, low = lowest(P, pos);
      // and of the item's first and last row
      const int pos0 = w.len + item_row / P.group;
      const int pos1 = w.len + (item_row + w.rows - 1) / P.group;
      const int low0 = lowest(P, pos0), low1 = lowest(P, pos1);
      const float slope = kMod && P.slopes ? P.slopes[w.h * P.group + g] * 1.4426950408889634f : 0.0f;
      uint32_t* odd = s.odd[item & 1];
      int taken[2] = {0, 0};  // tiles of this item that each stream took
      float m = -INFINITY, l = 0.0f;  // m: the maximum that O and l were taken with

      for (int t = w.t0; t < w.t1; t++) {
        if (pair) {
          taken[0]++;
          taken[1]++;
        } else {
          // by the item's own count, so that a row's sums do not depend on what ran before
          taken[(t - w.t0) & 1]++;
          if (((t - w.t0) & 1) != st) continue;
        }
        if (!__all_sync(kFullMask, barrier_wait(smem_of(&s.s_full[st]), scored & 1, gave_up))) break;
        const int key0 = w.tile(t) * kKeys;
        // holds keys that not every row sees
        const bool mixed = !(key0 + kKeys <= w.prefix || (key0 >= low1 && key0 + kKeys - 1 <= pos0));
        if (mixed && (!pair || st == 0)) {
          // (Only now that the scores are there: a wait tells phases apart by their parity,
          // so the copy before this one in the same stage must be known to have landed.)
          // A value that is not finite would pass through a weight of 0 into rows that do
          // not see its key: it becomes 0 here and comes back, at the end, for those that do.
          // (And what lies where nobody sees a key is whatever was there.)
          const uint32_t job = jobs + S::value_job(pair, t - w.t0, w.t1 - w.t0), stage = job % kStages;
          if (!__all_sync(kFullMask, barrier_wait(smem_of(&s.kv_full[stage]), job / kStages & 1, gave_up)))
            break;
          char* v = smem + S::kStageAt + stage * S::kTileBytes;
          bool changed = false;
          for (int e = quarter * 32 + lane; e < kKeys * (DP / 8); e += 128) {
            const int r = e / (DP / 8), p = e % (DP / 8), key = key0 + r;
            if (key < w.prefix || (key >= low1 && key <= pos0)) continue;  // all rows see it
            uint4* place = reinterpret_cast<uint4*>(v + (p / 8) * (kKeys * 128) + r * 128 + (p % 8) * 16);
            if (key > pos1 || key < low0) {  // nobody does
              *place = make_uint4(0, 0, 0, 0);
              changed = true;
              continue;
            }
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
              const int bit = key > pos0 ? key - pos0 - 1 : 32 * kEdge + key - low0;
              atomicOr(odd + bit / 32, 1u << bit % 32);
              changed = true;
            }
          }
          if (changed) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        __syncwarp();
        tmem_fence_after();
        const bool first = taken[st] == 1;
        if (working) {
          uint32_t x[kKeys];
          tmem_load128(tS[st] + lanes, x);
          if (kMod) {
            if (P.cap_log2 > 0.0f) {
              // cap tanh z = cap (1 - 2 / (1 + e^2z)): 2^-22 of the cap off, whatever z is
#pragma unroll
              for (int e = 0; e < kKeys; e++)
                x[e] = __float_as_uint(fmaf(
                    rcp_of(exp2_of(__uint_as_float(x[e]) * P.cap_turn) + 1.0f), -2.0f * P.cap_log2, P.cap_log2));
            } else {
#pragma unroll
              for (int e = 0; e < kKeys; e++) x[e] = __float_as_uint(__uint_as_float(x[e]) * c);
            }
            if (P.slopes) {
              const float from = static_cast<float>(key0 - pos);
#pragma unroll
              for (int e = 0; e < kKeys; e++)
                x[e] = __float_as_uint(fmaf(-slope, fabsf(from + e), __uint_as_float(x[e])));
            }
          }
          if (mixed) {
#pragma unroll
            for (int k = 0; k < kKeys; k += 32) {
              const int from = key0 + k;
              const uint32_t seen =
                  bits_below(w.prefix - from) | (bits_below(pos + 1 - from) & ~bits_below(low - from));
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
          float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
          if (!kMod) top *= c;
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
              const uint64_t xs = pair_of(x[k + e], x[k + e + 1]);
              const float2 y = halves_of(kMod ? add2(xs, shift2) : fma2(xs, c2, shift2));
              const float a = exp2_of(y.x), b = exp2_of(y.y);
              sums[e / 2 % 2] =
                  add2(sums[e / 2 % 2], pair_of(__float_as_uint(a), __float_as_uint(b)));
              // the weights' one rounding, to the type of the values they meet: the MMA takes
              // both operands in one 16-bit type.  (The sum has them as they are.)
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
      uint32_t odd_rows[2 * kEdge];
      bool fix = false;
#pragma unroll
      for (int k = 0; k < 2 * kEdge; k++) {
        odd_rows[k] = odd[k];
        fix |= odd_rows[k] != 0;
      }
      const float2 other = s.stats[st ^ 1][row];
      if (tid < 2 * kEdge) s.odd[(item & 1) ^ 1][tid] = 0;
      barrier_wait(smem_of(&s.item_checked[items % kItems]), items / kItems & 1, gave_up);
      const bool bad = __any_sync(kFullMask, given.bad != 0 || *gave_up);  // unchecked is bad
      // Only a checked request's pages are followed.  (Of a flagged one a box may not have
      // been copied, and what its place in the ring held before may look like such values.)
      fix = fix && !bad;
      __syncwarp();
      done_item();
      // A pair: this stream's rows, all columns; else half of the columns of both streams' sum
      const int my_rows = w.rows - first_row;
      if (quarter * 32 < my_rows && !(bad && !w.begins)) {
        float weight[2] = {1.0f, 1.0f};
        if (!pair) {
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
        const bool whole = w.pieces == 1 || bad;  // of a flagged request the first piece clears the rows
        const float inv = 1.0f / l;
        const bool mine = row < my_rows;
        uint16_t* out = P.out.data + (w.first + static_cast<int64_t>(token)) * P.out.node_stride +
                        (w.h * P.group + g) * P.out.head_stride;
        const int64_t slot = 2 * static_cast<int>(blockIdx.x) + w.begins;
        float4* part = P.ws.parts + slot * (DP / 4) * P.part_rows + first_row + row;
        const int cols = pair ? DP : DP / 2, col0 = pair ? 0 : st * cols;
#pragma unroll 1
        for (int k = 0; k < cols; k += 32) {
          float o[32];
          uint32_t x[32];
          if (pair) {
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
          if (mine && fix) {
#pragma unroll 1
            for (int word = 0; word < 2 * kEdge; word++) {
              uint32_t left = 0;
#pragma unroll
              for (int i = 0; i < 2 * kEdge; i++)
                if (i == word) left = odd_rows[i];
              for (; left; left &= left - 1) {
                const int bit = 32 * word + __ffs(left) - 1;
                const int key = bit < 32 * kEdge ? pos0 + 1 + bit : low0 + bit - 32 * kEdge;
                if (key > pos || key < low) continue;
                const uint16_t* v = C.v + C.slot(w.b, key) + w.h * C.head_stride;
#pragma unroll
                for (int e = 0; e < 32; e++) {
                  const int d = col0 + k + e;
                  if (d >= C.head_dim) continue;
                  const uint32_t bits = v[d];
                  if ((bits & kExp) == kExp) o[e] += E::unpack(bits).x;
                }
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
        if (!whole && mine && (pair || st == 0))
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

template <class E, int DP, bool kMod>
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

// One translation unit for each type of the cache.
template <class E>
cudaError_t run(const Params& P, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream);

template <class E>
cudaError_t run_any(const Params& P, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
  const bool mod = P.cap_log2 > 0.0f || P.slopes;
  if (P.cache.head_dim <= 64)
    return mod ? launch<E, 64, true>(P, k, v, stream) : launch<E, 64, false>(P, k, v, stream);
  return mod ? launch<E, 128, true>(P, k, v, stream) : launch<E, 128, false>(P, k, v, stream);
}

}  // namespace specv_chunk
