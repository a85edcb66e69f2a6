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
// and O is rescaled only when the maximum has risen by more than 2^8, which
// no result shows: m is whatever both O and the sum l were taken with.
//
// The work is the list of (request, key head, row tile, 128-key tile), cut
// into equal runs, one to a CTA and a CTA to an SM, so ragged lengths and few
// requests fill the machine alike.  A row tile whose keys one CTA has whole is
// written out; pieces leave (m, l, O) in the workspace for combine_kernel.
//
// Two streams share an SM, each with its S and O in TMEM and its four softmax
// warps: with up to 128 rows they take the key tiles in turn and are joined
// at the end (kPair false), with more they are two row tiles on the same keys
// (kPair true).  One thread issues the MMAs, four warps the copies.

#include <type_traits>

#include "cache.cuh"

using namespace specv_cache_ops;

namespace {

constexpr int kKeys = 128;     // keys of a tile
constexpr int kRows = 128;     // query rows of a stream
constexpr int kMaxCtas = 152;  // SMs of a GB300
constexpr int kLoadWarps = 4;
constexpr int kLoadWarp = 8;  // the first of them
constexpr int kMmaWarp = 12;  // the last three warps of its warpgroup have no work
constexpr int kThreads = 512;
// Registers a thread of each warpgroup: 2 * 200 + 64 + 48 = 512 = 4 * 128, what
// the block is launched with.  The softmax keeps a row of scores in them.
#define SPECV_REGS_SOFTMAX "200"
#define SPECV_REGS_LOAD "64"
#define SPECV_REGS_MMA "48"
constexpr float kRise = 8.0f;  // log2 of how far a maximum may rise before O is rescaled

// ----------------------------------------------------------------- prepare

constexpr int kPrepThreads = 128;

// What the attention kernel reads of a request (0 nodes where it is flagged).
struct Plan {
  int32_t* len;       // [B] verified tokens
  int32_t* nodes;     // [B]
  uint64_t* visible;  // [B][kMaxNodes] bit j: node sees node j
  int64_t* share;     // units of a CTA's run
  int4* starts;       // [ctas] request, head, row tile and key tile where a CTA begins
  float* parts;       // [2 ctas][rows][dim] pieces' O ...
  float2* stats;      // [2 ctas][rows]      ... and their m c and l
};

__global__ void __launch_bounds__(kPrepThreads) prepare_kernel(const Cache C, const int32_t* parents,
                                                               const int32_t* n_nodes, int N,
                                                               Plan plan, const Rows out,
                                                               int q_heads, int32_t* status) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
  const bool bad_page = !s_bad && bad_pages(C, b, 0, s_len + s_n, tid, kPrepThreads);
  const bool any = __syncthreads_or(bad_page);
  if (tid < 32) {
    if (any) t.bad |= SPECV_DEV_BAD_CACHE;
    if (!t.bad) {
      uint64_t bits[2];
      ancestors(t, lane, bits);
      plan.visible[static_cast<int64_t>(b) * kMaxNodes + lane] = bits[0];
      plan.visible[static_cast<int64_t>(b) * kMaxNodes + lane + 32] = bits[1];
    }
    if (lane == 0) {
      plan.len[b] = t.bad ? 0 : t.len;
      plan.nodes[b] = t.bad ? 0 : t.n;
      status[b] = static_cast<int32_t>(t.bad);
    }
  }
  if (s_bad || any) {  // a flagged request's rows become 0
    const int n = s_n ? s_n : N, words = C.head_dim / 8;
    for (int e = tid; e < n * q_heads * words; e += kPrepThreads) {
      const int i = e / (q_heads * words), h = e / words % q_heads, d = e % words * 8;
      *reinterpret_cast<uint4*>(out.data + b * out.batch_stride + i * out.node_stride +
                                h * out.head_stride + d) = make_uint4(0, 0, 0, 0);
    }
  }
}

// ------------------------------------------------------------- PTX wrappers

__device__ __forceinline__ uint32_t smem_of(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void barrier_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void barrier_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool barrier_try(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done;
}

__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

// Waits for a phase, two seconds at most: then, and from then on in the whole
// CTA, nothing waits any more.  The roles run their loops out (every address
// they form is in bounds whatever the data), and the request is flagged.
__device__ __forceinline__ void barrier_wait_slow(uint32_t bar, uint32_t parity, volatile int* gave_up) {
  const uint64_t start = now_ns();
  while (!barrier_try(bar, parity)) {
    if (*gave_up) return;
    if (now_ns() - start > 2000000000ull) {
      *gave_up = 1;
      return;
    }
  }
}

__device__ __forceinline__ void barrier_wait(uint32_t bar, uint32_t parity, volatile int* gave_up) {
  if (!barrier_try(bar, parity)) barrier_wait_slow(bar, parity, gave_up);
}

__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from),
               "r"(real ? 16 : 0)
               : "memory");
}

// Arrives on the barrier when this thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tmem_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Shared-memory operand with 128-byte swizzle: rows of 128 bytes, eight of
// them a 1024-byte group.  The low word holds the address and `lead`, the
// distance of the next 64 columns where the operand's contiguous dimension is
// not the summed one; a step along the operand is an addition to it.
__device__ __forceinline__ uint32_t operand_low(uint32_t at, uint32_t lead) {
  return (at & 0x3ffff) >> 4 | (lead >> 4) << 16;
}
constexpr uint32_t kOperandHigh = 1024 >> 4 | 1u << 14 | 2u << 29;

template <bool kAdd>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_low, uint32_t b_low, uint32_t idesc) {
  asm volatile(
      "{\n .reg .b64 a, b;\n .reg .pred p;\n"
      " mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %3};\n setp.ne.u32 p, %5, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n}" ::"r"(d),
      "r"(a_low), "r"(b_low), "r"(kOperandHigh), "r"(idesc), "n"(kAdd ? 1 : 0)
      : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_low, uint32_t idesc,
                                       uint32_t add) {
  asm volatile(
      "{\n .reg .b64 b;\n .reg .pred p;\n"
      " mov.b64 b, {%2, %3};\n setp.ne.u32 p, %5, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}" ::"r"(d),
      "r"(a), "r"(b_low), "r"(kOperandHigh), "r"(idesc), "r"(add)
      : "memory");
}

__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}

#define SPECV_R8(x, i)                                                                   \
  "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3]), "=r"(x[i + 4]),            \
      "=r"(x[i + 5]), "=r"(x[i + 6]), "=r"(x[i + 7])
#define SPECV_R32(x, i) \
  SPECV_R8(x, i), SPECV_R8(x, i + 8), SPECV_R8(x, i + 16), SPECV_R8(x, i + 24)
#define SPECV_I8(x, i)                                                                   \
  "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3]), "r"(x[i + 4]), "r"(x[i + 5]),  \
      "r"(x[i + 6]), "r"(x[i + 7])

// 32 columns of this warp's 32 lanes, a register to a column, waited for.
__device__ __forceinline__ void tmem_load32(uint32_t at, uint32_t (&x)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
      "%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : SPECV_R32(x, 0)
      : "r"(at)
      : "memory");
}

// 128 columns, waited for.
__device__ __forceinline__ void tmem_load128(uint32_t at, uint32_t (&x)[128]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%128];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%129];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,"
      "%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95}, [%130];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,"
      "%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%131];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : SPECV_R32(x, 0), SPECV_R32(x, 32), SPECV_R32(x, 64), SPECV_R32(x, 96)
      : "r"(at), "r"(at + 32), "r"(at + 64), "r"(at + 96)
      : "memory");
}

// 16 columns, waited for.
__device__ __forceinline__ void tmem_load16(uint32_t at, uint32_t (&x)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : SPECV_R8(x, 0), SPECV_R8(x, 8)
      : "r"(at)
      : "memory");
}

__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t (&x)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::SPECV_I8(x, 0),
      SPECV_I8(x, 8), "r"(at)
      : "memory");
}

__device__ __forceinline__ void tmem_store_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Two 32-bit operations in one instruction, each rounded as by itself.
__device__ __forceinline__ uint64_t pair_of(uint32_t lo, uint32_t hi) {
  uint64_t p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "r"(lo), "r"(hi));
  return p;
}
__device__ __forceinline__ float2 halves_of(uint64_t p) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
  return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// --------------------------------------------------------------- attention

struct AttnParams {
  Cache cache;
  Rows q, out;
  Plan plan;
  int32_t* status;
  int B, q_heads, group;  // group: query heads to a key head
  float scale_log2;
};

template <int DP, bool kPair> struct Shape {
  static constexpr int kTileBytes = kKeys * DP * 2;  // of keys, of values or of queries
  static constexpr int kStages = DP == 128 ? 5 : 10;
  static constexpr int kRowTile = kPair ? 2 * kRows : kRows;
  // shared memory: queries (two tiles: both row tiles, or this and the next item's), stages,
  // then the barriers and what the warps tell one another
  static constexpr int kStageAt = 2 * kTileBytes;
  static constexpr int kTailAt = kStageAt + kStages * kTileBytes;
};

struct Tail {
  uint64_t kv_full[10], kv_empty[10], q_full[2], q_empty[2], s_full[2], o_full[2];
  uint64_t p_full[2][2];   // by stream and half of the keys
  uint64_t odd_values[2];  // nodes whose values were not finite, by parity of the item
  int64_t base;            // work units before request `first`
  int64_t total;
  int first;
  int gave_up;
  uint32_t tmem;
  float2 stats[2][kRows];
};

// The work units (128-key tiles of a row tile of a key head) of request b.
template <int kRowTile>
__device__ __forceinline__ int64_t units_of(const AttnParams& P, int b, int& tiles, int& row_tiles) {
  const int n = P.plan.nodes[b];
  tiles = n ? (P.plan.len[b] + n + kKeys - 1) / kKeys : 0;
  row_tiles = (n * P.group + kRowTile - 1) / kRowTile;
  return static_cast<int64_t>(tiles) * row_tiles * P.cache.heads;
}

// A CTA's run of units, item by item (an item: all key tiles of a row tile).
template <int kRowTile> struct Walk {
  int64_t at, end, base, units;
  int b, tiles, row_tiles;
  // the current item, and which of its key tiles are this CTA's
  int h, row_tile, t0, t1, len, n;

  __device__ __forceinline__ void start(const AttnParams& P, const Tail& s, int64_t share) {
    at = static_cast<int64_t>(blockIdx.x) * share;
    end = min(at + share, s.total);
    b = s.first;
    base = s.base;
    if (at < end) units = units_of<kRowTile>(P, b, tiles, row_tiles);
  }
  __device__ __forceinline__ bool next(const AttnParams& P) {
    if (at >= end) return false;
    while (at >= base + units) {
      base += units;
      units = units_of<kRowTile>(P, ++b, tiles, row_tiles);
    }
    const int64_t off = at - base;
    const int64_t item = off / tiles;
    t0 = static_cast<int>(off - item * tiles);
    h = static_cast<int>(item / row_tiles);
    row_tile = static_cast<int>(item - static_cast<int64_t>(h) * row_tiles);
    t1 = static_cast<int>(min(static_cast<int64_t>(tiles), t0 + (end - at)));
    len = P.plan.len[b];
    n = P.plan.nodes[b];
    at += t1 - t0;
    return true;
  }
  __device__ __forceinline__ int rows(int group) const { return n * group - row_tile * kRowTile; }
};

// Bits of the 32 columns from `first` (a key's number less len): which of them
// a row sees whose nodes are `visible`.
__device__ __forceinline__ uint32_t seen_of(int first, uint64_t visible) {
  if (first <= -32) return ~0u;
  if (first < 0) return ~(~0u << -first) | static_cast<uint32_t>(visible) << -first;
  return first < 64 ? static_cast<uint32_t>(visible >> first) : 0u;
}

template <class E, int DP, bool kPair>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(const AttnParams P) {
  using S = Shape<DP, kPair>;
  constexpr int kStages = S::kStages;
  // weights in f16 go below 2^-14, where its steps stop shrinking: taken 2^7 larger
  // they reach 2^15 at most (2^kRise more than the maximum's)
  constexpr float kLift = std::is_same<E, F16>::value ? 7.0f : 0.0f;
  extern __shared__ __align__(1024) char smem[];
  Tail& s = *reinterpret_cast<Tail*>(smem + S::kTailAt);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  const uint32_t base = smem_of(smem);
  const Cache& C = P.cache;

  if (tid == 0) {
    for (int i = 0; i < kStages; i++) {
      barrier_init(smem_of(&s.kv_full[i]), 32 * kLoadWarps);
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
    s.gave_up = 0;
    s.first = 0;
    s.base = 0;
    s.total = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_of(&s.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = s.tmem;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // Where this CTA's run begins: the units of all requests, then the request
  // that holds the first of this CTA's.
  int64_t share;
  {
    int64_t mine = 0;
    int tiles, row_tiles;
    for (int b = tid; b < P.B; b += kThreads) mine += units_of<S::kRowTile>(P, b, tiles, row_tiles);
    atomicAdd(reinterpret_cast<unsigned long long*>(&s.total), static_cast<unsigned long long>(mine));
    __syncthreads();
    share = (s.total + gridDim.x - 1) / gridDim.x;
    const int64_t want = static_cast<int64_t>(blockIdx.x) * share;
    if (warp == 0 && want < s.total) {
      int64_t before = 0;
      for (int b0 = 0; b0 < P.B; b0 += 32) {
        const int64_t u =
            b0 + lane < P.B ? units_of<S::kRowTile>(P, b0 + lane, tiles, row_tiles) : 0;
        int64_t upto = u;
        for (int o = 1; o < 32; o *= 2) {
          const int64_t x = __shfl_up_sync(kFullMask, upto, o);
          if (lane >= o) upto += x;
        }
        if (want >= before + upto - u && want < before + upto) {
          s.first = b0 + lane;
          s.base = before + upto - u;
        }
        before += __shfl_sync(kFullMask, upto, 31);
        if (want < before) break;
      }
    }
    __syncthreads();
  }
  Walk<S::kRowTile> w;
  w.start(P, s, share);

  const uint32_t tS[2] = {tmem, tmem + 128};
  const uint32_t tO[2] = {tmem + 256, tmem + 256 + DP};
  volatile int* gave_up = &s.gave_up;

  if (warp >= kLoadWarp && warp < kMmaWarp) {
    // ------------------------------------------------------------- copies
    asm volatile("setmaxnreg.dec.sync.aligned.u32 " SPECV_REGS_LOAD ";");
    // Copies of 16 bytes, so that pages of any size and strides of any kind will
    // do; places without a key (behind the last, past the head) become 0.
    constexpr int kPieces = DP / 8;            // 16-byte pieces of a row
    constexpr int kRowsAtOnce = 32 / kPieces;  // rows of one warp instruction
    const int lw = warp - kLoadWarp, piece = lane % kPieces, sub = lane / kPieces;
    const bool inside = piece * 8 < C.head_dim;
    uint32_t job = 0, item = 0;
    // 128-byte rows, their 16-byte pieces swapped by the row's number: rows
    // kRowsAtOnce apart, and sub < kRowsAtOnce, so r and sub set bits of their own
    const uint32_t lane_at = (piece / 8) * (kKeys * 128) + (32 * lw + sub) * 128;
    const uint32_t swap = (piece % 8) ^ sub;
    auto tile_copy = [&](uint32_t to, const uint16_t* from, int64_t off) {
      // this lane's row is 32 lw + lane of the tile, at from + off (off < 0: none)
#pragma unroll
      for (int r = 0; r < 32; r += kRowsAtOnce) {
        const int64_t o = __shfl_sync(kFullMask, off, r + sub);
        const bool ok = o >= 0 && inside;
        copy16(to + lane_at + r * 128 + (swap ^ (r % 8)) * 16, from + (ok ? o + piece * 8 : 0), ok);
      }
    };
    while (w.next(P)) {
      const int q_buffer = kPair ? 0 : item & 1;
      const uint32_t q_use = kPair ? item : item / 2;
      barrier_wait(smem_of(&s.q_empty[q_buffer]), (q_use & 1) ^ 1, gave_up);
#pragma unroll
      for (int half = 0; half < (kPair ? 2 : 1); half++) {
        const int row = half * kRows + 32 * lw + lane;
        const bool real = row < w.rows(P.group);
        const int at = w.row_tile * S::kRowTile + (real ? row : 0);
        const int node = at / P.group, g = at - node * P.group;
        const int64_t off = w.b * P.q.batch_stride + node * P.q.node_stride +
                            (w.h * P.group + g) * P.q.head_stride;
        tile_copy(base + (kPair ? half : q_buffer) * S::kTileBytes, P.q.data, real ? off : -1);
      }
      copies_arrive(smem_of(&s.q_full[q_buffer]));
      item++;
      const int keys = w.len + w.n;
      // A lane's key of a tile: its page's number is read a tile ahead of its use.
      const int32_t* table = C.page_table + static_cast<int64_t>(w.b) * C.table_stride;
      auto key_of = [&](int t) { return t * kKeys + 32 * lw + lane; };
      auto page_of = [&](int t) {
        const int key = key_of(t);
        return t < w.t1 && key < keys ? table[key / C.page_size] : -1;
      };
      int page = page_of(w.t0), page_next = page_of(w.t0 + 1);
      for (int t = w.t0; t < w.t1; t++) {
        const int64_t off = page < 0 ? static_cast<int64_t>(-1)
                                     : page * C.page_stride +
                                           key_of(t) % C.page_size * C.row_stride +
                                           w.h * C.head_stride;
        page = page_next;
        page_next = page_of(t + 2);
#pragma unroll
        for (int kv = 0; kv < 2; kv++, job++) {
          const uint32_t stage = job % kStages, use = job / kStages;
          barrier_wait(smem_of(&s.kv_empty[stage]), (use & 1) ^ 1, gave_up);
          tile_copy(base + S::kStageAt + stage * S::kTileBytes, kv ? C.v : C.k, off);
          copies_arrive(smem_of(&s.kv_full[stage]));
        }
      }
    }
    // The MMAs' last arrivals must find this CTA's shared memory.
    for (int i = 0; i < kStages; i++, job++)
      barrier_wait(smem_of(&s.kv_empty[job % kStages]), (job / kStages & 1) ^ 1, gave_up);
    for (int i = 0; i < (kPair ? 1 : 2); i++, item++)
      barrier_wait(smem_of(&s.q_empty[kPair ? 0 : item & 1]), ((kPair ? item : item / 2) & 1) ^ 1,
                   gave_up);
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= kMmaWarp) {
    // --------------------------------------------------------------- MMAs
    asm volatile("setmaxnreg.dec.sync.aligned.u32 " SPECV_REGS_MMA ";");
    constexpr uint32_t kType = std::is_same<E, Bf16>::value ? 1 : 0;
    constexpr uint32_t kIdesc = 1u << 4 | kType << 7 | kType << 10 | (kRows >> 4) << 24;
    constexpr uint32_t kIdescS = kIdesc | (kKeys >> 3) << 17;
    constexpr uint32_t kIdescO = kIdesc | 1u << 16 | (DP >> 3) << 17;
    if (warp == kMmaWarp && lane == 0) {
      const int steps = (C.head_dim + 15) / 16;
      uint32_t tile = 0, item = 0;       // key tiles and items so far
      uint32_t weighted[2] = {0, 0};  // O updates of each stream so far
      auto stage_at = [&](uint32_t job) { return base + S::kStageAt + job % kStages * S::kTileBytes; };
      auto kv_wait = [&](uint32_t job) {
        barrier_wait(smem_of(&s.kv_full[job % kStages]), job / kStages & 1, gave_up);
        // the copies wrote through the generic proxy, the MMA reads through the other
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      };
      auto qk = [&](int st, uint32_t q_at, uint32_t k_at) {
        const uint32_t a = operand_low(q_at, 16), b = operand_low(k_at, 16);
        mma_ss<false>(tS[st], a, b, kIdescS);
#pragma unroll
        for (int k = 1; k < DP / 16; k++) {
          const uint32_t step = ((k / 4) * (kKeys * 128) + (k % 4) * 32) >> 4;
          if (k < steps) mma_ss<true>(tS[st], a + step, b + step, kIdescS);
        }
        mma_commit(smem_of(&s.s_full[st]));
      };
      auto pv = [&](int st, uint32_t v_at, bool first) {
        const uint32_t b = operand_low(v_at, kKeys * 128);
#pragma unroll
        for (int half = 0; half < 2; half++) {
          barrier_wait(smem_of(&s.p_full[st][half]), weighted[st] & 1, gave_up);
          tmem_fence_after();
#pragma unroll
          for (int k = half * kKeys / 32; k < (half + 1) * kKeys / 32; k++)
            mma_ts(tO[st], tS[st] + 8 * k, b + (k * 2048 >> 4), kIdescO, k > 0 || !first);
        }
        mma_commit(smem_of(&s.o_full[st]));
        weighted[st]++;
      };
      // the update that is due: a tile's values wait until the next tile's scores are issued
      bool due = false, due_first = false;
      bool due_second = false;  // kPair: the item has rows for stream 1
      auto last_pair = [&](uint32_t v_job) {
        kv_wait(v_job);
        pv(0, stage_at(v_job), due_first);
        if (due_second) pv(1, stage_at(v_job), due_first);
        mma_commit(smem_of(&s.kv_empty[v_job % kStages]));
      };
      while (w.next(P)) {
        const int q_buffer = kPair ? 0 : item & 1;
        const uint32_t q_use = kPair ? item : item / 2;
        const bool second = kPair && w.rows(P.group) > kRows;
        bool started[2] = {false, false};
        if (kPair && due) {  // the queries have one buffer: nothing to issue before they are there
          last_pair(2 * tile - 1);
          due = false;
        }
        barrier_wait(smem_of(&s.q_full[q_buffer]), q_use & 1, gave_up);
        for (int t = w.t0; t < w.t1; t++, tile++) {
          const uint32_t k_job = 2 * tile, v_job = 2 * tile - 1;  // this tile's keys, the last's values
          if (kPair) {
            if (due) {
              kv_wait(v_job);
              pv(0, stage_at(v_job), due_first);
            }
            kv_wait(k_job);
            qk(0, base, stage_at(k_job));
            if (due && due_second) pv(1, stage_at(v_job), due_first);
            if (due) mma_commit(smem_of(&s.kv_empty[v_job % kStages]));
            if (second) qk(1, base + S::kTileBytes, stage_at(k_job));
            mma_commit(smem_of(&s.kv_empty[k_job % kStages]));
            due_first = t == w.t0;
            due_second = second;
          } else {
            const int st = tile & 1;
            kv_wait(k_job);
            qk(st, base + q_buffer * S::kTileBytes, stage_at(k_job));
            mma_commit(smem_of(&s.kv_empty[k_job % kStages]));
            if (due) {
              kv_wait(v_job);
              pv(st ^ 1, stage_at(v_job), due_first);
              mma_commit(smem_of(&s.kv_empty[v_job % kStages]));
            }
            due_first = !started[st];
            started[st] = true;
          }
          due = true;
        }
        mma_commit(smem_of(&s.q_empty[q_buffer]));
        item++;
      }
      if (due) {
        const uint32_t v_job = 2 * tile - 1;
        if (kPair) {
          last_pair(v_job);
        } else {
          kv_wait(v_job);
          pv((tile - 1) & 1, stage_at(v_job), due_first);
          mma_commit(smem_of(&s.kv_empty[v_job % kStages]));
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 " SPECV_REGS_SOFTMAX ";");
    const int st = warp / 4, quarter = warp % 4;
    const int row = quarter * 32 + lane;  // of the stream's tile
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const float c = P.scale_log2;
    uint32_t tile = 0, item = 0, scores[2] = {0, 0};  // scores: tiles of each stream so far
    bool told = false;
    while (w.next(P)) {
      const int rows = w.rows(P.group);
      const int first_row = kPair ? st * kRows : 0;
      const bool second = !kPair || rows > kRows;
      const bool working = first_row + quarter * 32 < rows;  // this warp has rows
      const int at = w.row_tile * S::kRowTile + min(first_row + row, rows - 1);
      const int node = at / P.group, g = at - node * P.group;
      const uint64_t visible = P.plan.visible[static_cast<int64_t>(w.b) * kMaxNodes + node];
      const int keys = w.len + w.n;
      uint64_t* odd = &s.odd_values[item & 1];
      int taken[2] = {0, 0};  // tiles of this item that each stream took
      float m = -INFINITY, l = 0.0f;  // m: the maximum that O and l were taken with, times c

      for (int t = w.t0; t < w.t1; t++, tile++) {
        if (kPair) {
          taken[0]++;
          if (second) taken[1]++;
          if (st == 1 && !second) continue;
        } else {
          taken[tile & 1]++;
          if ((tile & 1) != st) continue;
        }
        const bool mixed = (t + 1) * kKeys > w.len;  // holds keys that not every row sees
        if (mixed && (!kPair || st == 0)) {
          // A value that is not finite would pass through a weight of 0 into rows that do
          // not see its node: it becomes 0 here and comes back, at the end, for those that do.
          const uint32_t job = 2 * tile + 1, stage = job % kStages;
          barrier_wait(smem_of(&s.kv_full[stage]), job / kStages & 1, gave_up);
          char* v = smem + S::kStageAt + stage * S::kTileBytes;
          const int from = max(w.len - t * kKeys, 0), to = min(keys - t * kKeys, kKeys);
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
          if (changed) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        barrier_wait(smem_of(&s.s_full[st]), scores[st] & 1, gave_up);
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
            barrier_wait(smem_of(&s.o_full[st]), (scores[st] - 1) & 1, gave_up);
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
              // the weights' one rounding, to the type of the values they meet
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
        scores[st]++;
      }

      // The item's end: both streams' last updates, and what they know.
      if (!kPair) scores[st ^ 1] += taken[st ^ 1];
      else if (st == 0) scores[1] += taken[1];
      else scores[0] += taken[0];
#pragma unroll
      for (int k = 0; k < 2; k++)
        if (taken[k]) barrier_wait(smem_of(&s.o_full[k]), (scores[k] - 1) & 1, gave_up);
      tmem_fence_after();
      s.stats[st][row] = make_float2(m, l);
      asm volatile("bar.sync 1, 256;" ::: "memory");
      const uint64_t fix = *odd & visible;
      const float2 other = s.stats[st ^ 1][row];
      if (tid == 0) s.odd_values[(item & 1) ^ 1] = 0;
      if (*gave_up && !told) {
        told = true;
        if (tid == 0) atomicOr(P.status + w.b, SPECV_DEV_TIMEOUT);
      }
      // kPair: this stream's rows, all columns; else half of the columns of both streams' sum
      const int my_rows = rows - first_row;
      if (quarter * 32 < my_rows) {
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
        const bool whole = w.t0 == 0 && w.t1 == w.tiles;
        const float inv = 1.0f / l;
        const bool mine = row < my_rows;
        uint16_t* out = P.out.data + w.b * P.out.batch_stride + node * P.out.node_stride +
                        (w.h * P.group + g) * P.out.head_stride;
        const int slot = 2 * blockIdx.x + (w.t0 == 0);
        const int64_t part = static_cast<int64_t>(slot) * S::kRowTile + first_row + row;
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
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              const int d = col0 + k + e;
              if (d < C.head_dim)
                *reinterpret_cast<uint4*>(out + d) =
                    make_uint4(E::pack(o[e] * inv, o[e + 1] * inv),
                               E::pack(o[e + 2] * inv, o[e + 3] * inv),
                               E::pack(o[e + 4] * inv, o[e + 5] * inv),
                               E::pack(o[e + 6] * inv, o[e + 7] * inv));
            }
          } else if (mine) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4*>(P.plan.parts + part * DP + col0 + k + e) =
                  make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
          __syncwarp();
        }
        if (!whole && mine && (kPair || st == 0)) P.plan.stats[part] = make_float2(m, l);
      }
      item++;
      tmem_fence_before();
      asm volatile("bar.sync 1, 256;" ::: "memory");
      tmem_fence_after();
    }
  }

  // Where this CTA began, for combine_kernel.
  if (tid == 0) {
    Walk<S::kRowTile> v;
    v.start(P, s, share);
    int4 at = make_int4(0, 0, 0, 0);
    if (v.next(P)) at = make_int4(v.b, v.h, v.row_tile, v.t0);
    P.plan.starts[blockIdx.x] = at;
    if (blockIdx.x == 0) *P.plan.share = share;
  }
  tmem_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// ----------------------------------------------------------------- combine

constexpr int kCombineWarps = 8;

// Joins the pieces of the items that runs of units cut.  Block x stands for the
// cut before CTA x's run; the first cut of an item joins all its pieces:
//   m = max m_i, O = sum 2^(m_i - m) O_i / sum 2^(m_i - m) l_i, in order.
// A warp has a row, a lane four of its columns.
template <class E, int DP, int kRowTile>
__global__ void __launch_bounds__(kCombineWarps * 32) combine_kernel(const AttnParams P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int cta = blockIdx.x + 1, lane = threadIdx.x & 31;
  const int4 at = P.plan.starts[cta];
  const int t0 = at.w;
  if (t0 == 0) return;  // no cut here
  const int row = blockIdx.y * kCombineWarps + threadIdx.x / 32;
  const int b = at.x, h = at.y, n = P.plan.nodes[b];
  const int flat = at.z * kRowTile + row;
  if (row >= kRowTile || flat >= n * P.group) return;
  // runs are of equal length: the one before began `share` units earlier
  const int4 before = P.plan.starts[cta - 1];
  if (before.x == b && before.y == h && before.z == at.z && before.w != 0) return;  // not the first
  const int tiles = (P.plan.len[b] + n + kKeys - 1) / kKeys;
  const int share = static_cast<int>(min(*P.plan.share, static_cast<int64_t>(INT_MAX)));
  const int pieces = 1 + (tiles - t0 - 1) / share + 1;
  auto index = [&](int i) {  // piece 0 ends CTA cta - 1's run, the others begin theirs
    const int slot = i == 0 ? 2 * (cta - 1) + 1 : 2 * (cta + i - 1);
    return static_cast<int64_t>(slot) * kRowTile + row;
  };
  float m = -INFINITY;
  for (int i = lane; i < pieces; i += 32) m = fmaxf(m, P.plan.stats[index(i)].x);
#pragma unroll
  for (int o = 16; o > 0; o /= 2) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, o));
  const int d = 4 * lane;
  float l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int i = 0; i < pieces; i++) {
    const float2 ml = P.plan.stats[index(i)];
    const float weight = ml.x == m ? 1.0f : exp2_of(ml.x - m);
    l = fmaf(weight, ml.y, l);
    if (d < DP) {
      const float4 x = *reinterpret_cast<const float4*>(P.plan.parts + index(i) * DP + d);
      o[0] = fmaf(weight, x.x, o[0]);
      o[1] = fmaf(weight, x.y, o[1]);
      o[2] = fmaf(weight, x.z, o[2]);
      o[3] = fmaf(weight, x.w, o[3]);
    }
  }
  if (d >= P.cache.head_dim) return;
  const float inv = 1.0f / l;
  const int node = flat / P.group, g = flat - node * P.group;
  *reinterpret_cast<uint2*>(P.out.data + b * P.out.batch_stride + node * P.out.node_stride +
                            (h * P.group + g) * P.out.head_stride + d) =
      make_uint2(E::pack(o[0] * inv, o[1] * inv), E::pack(o[2] * inv, o[3] * inv));
}

// ------------------------------------------------------------------- host

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

struct Layout {
  size_t nodes, visible, share, starts, stats, parts, total;
};

Layout layout(int B, int row_tile, int dim) {
  Layout w;
  w.nodes = align256(static_cast<size_t>(B) * 4);
  w.visible = w.nodes + align256(static_cast<size_t>(B) * 4);
  w.share = w.visible + align256(static_cast<size_t>(B) * kMaxNodes * 8);
  w.starts = w.share + 256;
  w.stats = w.starts + align256(kMaxCtas * sizeof(int4));
  w.parts = w.stats + align256(2 * kMaxCtas * sizeof(float2) * static_cast<size_t>(row_tile));
  w.total = w.parts + align256(2 * kMaxCtas * sizeof(float) * static_cast<size_t>(row_tile) * dim);
  return w;
}

int padded(int head_dim) { return head_dim <= 64 ? 64 : 128; }
bool paired(int N, int group) { return N * group > kRows; }

template <class E, int DP, bool kPair>
cudaError_t run(const AttnParams& P, int N, int ctas, cudaStream_t stream) {
  using S = Shape<DP, kPair>;
  constexpr int kSmem = S::kTailAt + static_cast<int>(sizeof(Tail));
  static_assert(kSmem <= 232448, "one CTA's shared memory");
  cudaError_t e = cudaFuncSetAttribute(attention_kernel<E, DP, kPair>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, attention_kernel<E, DP, kPair>, P);
  if (e != cudaSuccess || ctas == 1) return e;
  const int rows = N * P.group < S::kRowTile ? N * P.group : S::kRowTile;
  cfg.gridDim = dim3(ctas - 1, (rows + kCombineWarps - 1) / kCombineWarps);
  cfg.blockDim = dim3(kCombineWarps * 32);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, combine_kernel<E, DP, S::kRowTile>, P);
}

template <class E>
cudaError_t run_any(const AttnParams& P, bool pair, int dim, int N, int ctas, cudaStream_t stream) {
  if (dim == 64)
    return pair ? run<E, 64, true>(P, N, ctas, stream) : run<E, 64, false>(P, N, ctas, stream);
  return pair ? run<E, 128, true>(P, N, ctas, stream) : run<E, 128, false>(P, N, ctas, stream);
}

}  // namespace

extern "C" {

size_t specv_attention_workspace_bytes(int B, int N, int q_heads, int kv_heads, int head_dim) {
  if (B < 1 || B > SPECV_MAX_BATCH || N < 1 || N > SPECV_MAX_NODES || kv_heads < 1 ||
      q_heads < kv_heads || q_heads > 1024 || q_heads % kv_heads != 0 || head_dim < 8 ||
      head_dim > SPECV_MAX_HEAD_DIM || head_dim % 8 != 0)
    return 0;
  return layout(B, paired(N, q_heads / kv_heads) ? 2 * kRows : kRows, padded(head_dim)).total;
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
  const bool pair = paired(N, group);
  const int dim = padded(cache->head_dim);
  const Layout w = layout(B, pair ? 2 * kRows : kRows, dim);
  if (workspace_bytes < w.total) return SPECV_ERR_WORKSPACE;
  int device = 0, ctas = 0;
  if (cudaGetDevice(&device) != cudaSuccess ||
      cudaDeviceGetAttribute(&ctas, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
    return SPECV_ERR_CUDA;
  if (ctas > kMaxCtas) ctas = kMaxCtas;
  char* base = static_cast<char*>(workspace);
  const Plan plan{reinterpret_cast<int32_t*>(base),
                  reinterpret_cast<int32_t*>(base + w.nodes),
                  reinterpret_cast<uint64_t*>(base + w.visible),
                  reinterpret_cast<int64_t*>(base + w.share),
                  reinterpret_cast<int4*>(base + w.starts),
                  reinterpret_cast<float*>(base + w.parts),
                  reinterpret_cast<float2*>(base + w.stats)};
  const Cache C = to_cache(cache);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  prepare_kernel<<<B, kPrepThreads, 0, st>>>(C, parents, n_nodes, N, plan, to_rows(out), q_heads,
                                             status);
  const AttnParams P{C,       to_rows(q), to_rows(out), plan, status, B, q_heads, group,
                     scale * 1.4426950408889634f};
  const cudaError_t e = cache->dtype == SPECV_BF16 ? run_any<Bf16>(P, pair, dim, N, ctas, st)
                                                   : run_any<F16>(P, pair, dim, N, ctas, st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return SPECV_ERR_CUDA;
  }
  return launched();
}

}  // extern "C"
