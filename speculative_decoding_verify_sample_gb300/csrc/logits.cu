// Penalties for repeated tokens, biases and grammar masks on the logits of a
// drafted tree's (or chain's) rows: for a token of the row's text, c times in its
// generated part,
//
//   z <- (z > 0 ? z / rho : z rho) - freq c - pres  (the last two where c > 0),
//
// then z <- z + bias, and -inf where the mask has no bit.
//
// Bytes bound it: each row is read and written once (not read where the mask
// leaves nothing of 16 bytes), and what the text says is laid over the copy.
// Measured: 512 requests, two rows of 129,280 bf16 and texts of up to 4,001 tokens
// 94 us (4.4 TB/s of rows; mask and copy alone 64), 32 trees of up to 32 nodes
// over 128,256 entries 72 us (4.8 TB/s), one chain of five rows 6.1 us.  The rest is
// the text, which every chunk's block reads in whole before it can patch.

#include "cache.cuh"

using namespace specv_cache_ops;

namespace {

// A vocabulary entry's word: how often the text's generated part has it, and
constexpr uint32_t kInPrompt = 1u << 31;  // the prompt has it
constexpr uint32_t kBiased = 1u << 30;    // a bias names it
constexpr uint32_t kDrafted = 1u << 29;   // a drafted node's token is it
constexpr uint32_t kCount = kDrafted - 1;

struct Params {
  const char* in;
  char* out;
  int64_t batch_stride, row_stride, out_batch_stride, out_row_stride;  // elements
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* n_rows;
  const int32_t* history;
  int64_t history_stride;
  const int32_t* seq_lens;
  const int32_t* prompt_lens;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const int32_t* bias_tokens;
  const float* bias_values;
  const int32_t* allowed;
  int32_t* status;
  int R, V, L, num_bias;
  int rows;  // of a block
};

template <int DT> struct Elt;
template <> struct Elt<SPECV_F32> {
  using T = uint32_t;
  static constexpr uint32_t kNegInf = 0xff800000u;
  static __device__ float load(uint32_t w) { return __uint_as_float(w); }
  static __device__ uint32_t store(float x) { return __float_as_uint(x); }
};
template <> struct Elt<SPECV_BF16> {
  using T = uint16_t;
  static constexpr uint16_t kNegInf = 0xff80u;
  static __device__ float load(uint16_t w) { return __uint_as_float(static_cast<uint32_t>(w) << 16); }
  static __device__ uint16_t store(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
};

constexpr int kTokens = 512;  // tokens of the text that a warp counts at a time
constexpr int kFound = 160;   // of them in the chunk: four from each lane may follow 31 that wait
constexpr int kMaxRows = 8;     // rows of a block (32 nodes, 256 threads: 79 us; four 86, sixteen 84)

// What a block needs of one request's text, for its chunk of the vocabulary.
template <int kChunk, int kWarps> struct Text {
  uint32_t count[kChunk];
  uint64_t path[kMaxNodes];
  float bias[SPECV_MAX_BIAS];       // sums of the biases in this chunk ...
  uint16_t biased[SPECV_MAX_BIAS];  // ... and their entries
  int drafted[kMaxNodes];  // entry of node i's token, -1 where it is another chunk's
  int num_biased, touched, ticket, bad;
  uint32_t found[kWarps][kFound];  // by warp: tokens of the text that are in this chunk
  uint16_t list[8];  // touched entries: at most kChunk, and the text's, drafts' and biases' number
};

// How a row's elements lie against 16 bytes: every row begins there, rows
// begin anywhere but input and output alike, or not alike.
enum Layout { kAligned, kShifted, kSingle };

// -inf where keep's bit is 0.
template <int DT> __device__ __forceinline__ void mask_vec(uint4& v, uint32_t keep) {
  uint32_t* w = &v.x;
  if (DT == SPECV_F32) {
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (!(keep >> i & 1)) w[i] = 0xff800000u;
  } else {
#pragma unroll
    for (int i = 0; i < 2; i++) {
      // four bits to the tops of four bytes (the shifted copies do not meet), which
      // prmt then spreads over two bytes each
      const uint32_t tops = (keep >> 4 * i & 15u) * 0x10204080u;
      uint32_t lo, hi;
      asm("prmt.b32 %0, %1, 0, 0x9988;" : "=r"(lo) : "r"(tops));
      asm("prmt.b32 %0, %1, 0, 0xbbaa;" : "=r"(hi) : "r"(tops));
      w[2 * i] = (w[2 * i] & lo) | (0xff80ff80u & ~lo);
      w[2 * i + 1] = (w[2 * i + 1] & hi) | (0xff80ff80u & ~hi);
    }
  }
}

// A block takes kChunk vocabulary entries of one request, for P.rows of its
// rows.  It counts the text's tokens in this chunk in shared memory and lists
// the entries they touch.  Nearly every element is only masked and copied,
// whatever the text says, so the warps take first parts of the text and then
// segments of rows off one counter, and none waits for another.  Then the
// listed entries are computed from the input, one to a thread for two rows, and
// stored over the copies.
template <int DT, int kChunk, int kThreads, Layout kLayout>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) logits_kernel(const Params P) {
  using E = Elt<DT>;
  using T = typename E::T;
  constexpr int kVec = kLayout == kSingle ? 1 : 16 / sizeof(T);
  constexpr int kSegment = 1024;  // entries of a row that a warp copies at a time
  constexpr int kMine = kSegment / 32 / kVec;        // vectors of a segment a lane has
  constexpr int kFlight = kMine < 4 ? kMine : 4;     // ... in flight
  extern __shared__ __align__(16) char smem[];
  using S = Text<kChunk, kThreads / 32>;
  S& s = *reinterpret_cast<S*>(smem);

  const int tid = threadIdx.x, lane = tid & 31, b = blockIdx.y;
  const int c0 = blockIdx.x * kChunk, c1 = min(P.V, c0 + kChunk);
  const int given = P.n_rows ? P.n_rows[b] : P.R;
  const int total = P.seq_lens[b], prompt = P.prompt_lens ? P.prompt_lens[b] : 0;
  const float rho = P.repetition ? P.repetition[b] : 1.0f;
  const float freq = P.frequency ? P.frequency[b] : 0.0f;
  const float pres = P.presence ? P.presence[b] : 0.0f;
  for (int e = tid; e < kChunk / 4; e += kThreads)
    reinterpret_cast<uint4*>(s.count)[e] = make_uint4(0, 0, 0, 0);
  if (tid == 0) {
    s.num_biased = 0;
    s.touched = 0;
    s.ticket = 0;
    s.bad = 0;
  }
  const int n = given < 1 || given > P.R ? P.R : given;
  const int first_row = blockIdx.z * P.rows, last_row = min(n, first_row + P.rows);
  if (first_row >= last_row) return;
  __syncthreads();

  // Whoever finds an untouched word lists its entry.  Counts are whole numbers:
  // the order in which the threads add does not show.
  auto touch = [&](int e, uint32_t old) {
    if (old == 0) s.list[atomicAdd(&s.touched, 1)] = static_cast<uint16_t>(e);
  };
  const bool fits = total >= 0 && total <= P.L;
  if (tid < 32) {
    Tree t = read_tree(P.parents, P.n_rows, P.seq_lens, b, P.R, INT64_MAX, lane);
    if (!(t.bad & SPECV_DEV_BAD_TREE)) {
      bool bad_token = false;
#pragma unroll
      for (int k = 0; k < 2; k++) {
        const int i = lane + 32 * k;
        int at = -1;
        if (i >= 1 && i < t.n) {
          const int token = P.parents ? P.tokens[static_cast<int64_t>(b) * P.R + i]
                                      : P.tokens[static_cast<int64_t>(b) * (P.R - 1) + i - 1];
          bad_token |= token < 0 || token >= P.V;
          if (token >= c0 && token < c1) at = token - c0;
        }
        s.drafted[i] = at;
        if (at >= 0) touch(at, atomicOr(&s.count[at], kDrafted));
      }
      if (__any_sync(kFullMask, bad_token)) t.bad |= SPECV_DEV_BAD_TOKEN;
      // paths matter only where a drafted token is one of this chunk's
      if (__any_sync(kFullMask, s.drafted[lane] >= 0 || s.drafted[lane + 32] >= 0)) {
        uint64_t bits[2];
        ancestors(t, lane, bits);
        s.path[lane] = bits[0];
        s.path[lane + 32] = bits[1];
      }
    }
    if (total > P.L || prompt < 0 || prompt > total) t.bad |= SPECV_DEV_BAD_CACHE;
    if (!(rho > 0.0f) || !isfinite(rho) || !isfinite(freq) || !isfinite(pres))
      t.bad |= SPECV_DEV_BAD_PENALTY;
    if (lane == 0 && t.bad) atomicOr(&s.bad, static_cast<int>(t.bad));
  }
  bool bad_token = false;
  {
    const int32_t* names = P.bias_tokens + static_cast<int64_t>(b) * P.num_bias;
    const float* values = P.bias_values + static_cast<int64_t>(b) * P.num_bias;
    for (int i = tid; i < P.num_bias; i += kThreads) {
      const int token = names[i];
      bad_token |= token >= P.V;
      if (token < c0 || token >= c1) continue;
      // the first place that names a token adds up all of them, in their order
      float sum = 0.0f;
      bool first = true;
      for (int j = 0; j < P.num_bias; j++)
        if (names[j] == token) {
          if (j < i) first = false;
          sum = sum + values[j];
        }
      if (first) {
        const int at = atomicAdd(&s.num_biased, 1);
        s.biased[at] = static_cast<uint16_t>(token - c0);
        s.bias[at] = sum;
        touch(token - c0, atomicOr(&s.count[token - c0], kBiased));
      }
    }
  }
  auto take = [&]() {
    const int ticket = lane == 0 ? atomicAdd(&s.ticket, 1) : 0;
    return __shfl_sync(kFullMask, ticket, 0);
  };
  int ticket = take();
  const int parts = fits ? (total + kTokens - 1) / kTokens : 0;
  if (ticket < parts) {
    const int32_t* hist = P.history + b * P.history_stride;
    const bool vectors = reinterpret_cast<uintptr_t>(hist) % 16 == 0;
    unsigned largest = 0;
    // Of the text's tokens a small part is in this chunk: a warp gathers those
    // first, and counts them 32 at a time.  (Counting each where it is found took
    // three times the instructions: nearly always one of 32 lanes has one.)
    uint32_t* found = s.found[tid / 32];
    int waiting = 0;  // the same on every lane
    auto gather = [&](int i, int token) {
      const uint32_t e = token - c0;
      if (i < total) largest = max(largest, static_cast<unsigned>(token));
      const bool mine = i < total && e < static_cast<uint32_t>(c1 - c0);
      const uint32_t who = __ballot_sync(kFullMask, mine);
      if (mine) found[waiting + __popc(who & ((1u << lane) - 1))] = e | (i < prompt ? kInPrompt : 0);
      waiting += __popc(who);
    };
    auto count_found = [&](int most) {  // all but `most` at the front
      __syncwarp();
      while (waiting > most) {
        const int at = waiting - 1 - lane;
        if (at >= 0 && at >= waiting - 32) {
          const uint32_t word = found[at], e = word & ~kInPrompt;
          touch(e, word & kInPrompt ? atomicOr(&s.count[e], kInPrompt) : atomicAdd(&s.count[e], 1u));
        }
        waiting = max(waiting - 32, 0);
      }
      __syncwarp();
    };
    for (; ticket < parts; ticket = take()) {
      int4 t[kTokens / 128];
#pragma unroll
      for (int k = 0; k < kTokens / 128; k++) {
        const int i = ticket * kTokens + k * 128 + lane * 4;
        t[k] = make_int4(0, 0, 0, 0);
        if (vectors && i + 3 < total) {
          t[k] = *reinterpret_cast<const int4*>(hist + i);
        } else {
          if (i < total) t[k].x = hist[i];
          if (i + 1 < total) t[k].y = hist[i + 1];
          if (i + 2 < total) t[k].z = hist[i + 2];
          if (i + 3 < total) t[k].w = hist[i + 3];
        }
      }
#pragma unroll
      for (int k = 0; k < kTokens / 128; k++) {
        const int i = ticket * kTokens + k * 128 + lane * 4;
        gather(i, t[k].x);
        gather(i + 1, t[k].y);
        gather(i + 2, t[k].z);
        gather(i + 3, t[k].w);
        count_found(31);
      }
    }
    count_found(0);
    bad_token |= largest >= static_cast<unsigned>(P.V);
  }
  if (bad_token) atomicOr(&s.bad, SPECV_DEV_BAD_TOKEN);

  const T* in0 = reinterpret_cast<const T*>(P.in) + b * P.batch_stride;
  T* out0 = reinterpret_cast<T*>(P.out) + b * P.out_batch_stride;
  const int64_t words = (P.V + 31) / 32;
  auto mask_of = [&](int row) { return P.allowed + (static_cast<int64_t>(b) * P.R + row) * words; };

  // Copies and masks.  A segment's mask is read while the one before is copied.
  constexpr int kSegments = kChunk / kSegment;
  const int tickets = (last_row - first_row) * kSegments;
  struct Segment {
    int row, s0, s1;
  };
  auto segment_of = [&](int ticket, uint32_t (&keep)[kMine]) {
    ticket -= parts;
    Segment g{-1, 0, 0};
    if (ticket >= tickets) return g;
    g.row = first_row + ticket / kSegments;
    g.s0 = c0 + ticket % kSegments * kSegment;
    g.s1 = min(c1, g.s0 + kSegment);  // nothing left in the last chunk's last segments
    if (kLayout == kAligned && g.s1 - g.s0 == kSegment) {
#pragma unroll
      for (int u = 0; u < kMine; u++) {
        const int at = g.s0 + (u * 32 + lane) * kVec;
        keep[u] = P.allowed ? static_cast<uint32_t>(mask_of(g.row)[at >> 5]) >> (at & 31) : ~0u;
      }
    }
    return g;
  };
  uint32_t keep_next[kMine];
  Segment next = segment_of(ticket, keep_next);
  while (next.row >= 0) {
    const int row = next.row, s0 = next.s0, s1 = next.s1;
    uint32_t keep[kMine];
#pragma unroll
    for (int u = 0; u < kMine; u++) keep[u] = keep_next[u] & ((1u << kVec) - 1);
    const T* in = in0 + row * P.row_stride;
    T* out = out0 + row * P.out_row_stride;
    if (kLayout == kAligned && s1 - s0 == kSegment) {
      bool asked = false;
#pragma unroll
      for (int u0 = 0; u0 < kMine; u0 += kFlight) {
        uint4 data[kFlight];
#pragma unroll
        for (int u = 0; u < kFlight; u++)
          if (keep[u0 + u])  // where nothing is allowed there is nothing to read
            data[u] = *reinterpret_cast<const uint4*>(in + s0 + ((u0 + u) * 32 + lane) * kVec);
        if (!asked) {
          next = segment_of(take(), keep_next);
          asked = true;
        }
#pragma unroll
        for (int u = 0; u < kFlight; u++) {
          if (keep[u0 + u] != (1u << kVec) - 1) mask_vec<DT>(data[u], keep[u0 + u]);
          *reinterpret_cast<uint4*>(out + s0 + ((u0 + u) * 32 + lane) * kVec) = data[u];
        }
      }
    } else {
      const int32_t* mask = P.allowed ? mask_of(row) : nullptr;
      // vectors that begin before the segment and end behind it go by elements
      const int lead = kLayout == kSingle ? 0
                                          : static_cast<int>(reinterpret_cast<uintptr_t>(in + s0) /
                                                             sizeof(T) % kVec);
#pragma unroll 4
      for (int u = 0; u < kMine + (kVec > 1); u++) {
        const int at = s0 - lead + (u * 32 + lane) * kVec;
        const int from = max(at, s0), to = min(at + kVec, s1);
        if (from >= to) continue;
        uint32_t keep = (1u << kVec) - 1;
        if (mask) {
          uint64_t both = static_cast<uint32_t>(mask[from >> 5]);
          if ((to - 1) >> 5 != from >> 5) both |= static_cast<uint64_t>(mask[(to - 1) >> 5]) << 32;
          keep &= static_cast<uint32_t>(both >> (from & 31)) << (from - at);
        }
        if (kVec > 1 && to - from == kVec) {
          uint4 data;
          if (keep) data = *reinterpret_cast<const uint4*>(in + at);
          mask_vec<DT>(data, keep);
          *reinterpret_cast<uint4*>(out + at) = data;
        } else {
#pragma unroll
          for (int e = 0; e < kVec; e++)
            if (at + e >= from && at + e < to)
              out[at + e] = keep >> e & 1 ? in[at + e] : static_cast<T>(E::kNegInf);
        }
      }
      next = segment_of(take(), keep_next);
    }
  }
  __syncthreads();
  const int bad = s.bad;
  if (blockIdx.x == 0 && blockIdx.z == 0 && tid == 0) P.status[b] = bad;
  if (bad) {
    for (int row = first_row; row < last_row; row++)
      for (int t = c0 + tid; t < c1; t += kThreads)
        out0[row * P.out_row_stride + t] = static_cast<T>(E::kNegInf);
    return;
  }

  // The entries that the text, a draft or a bias touches.  (In place, the copy
  // left them as they were, or masked.)
  const int touched = s.touched, blocks = (touched + 31) / 32, pairs = (last_row - first_row + 1) / 2;
  for (int unit = tid / 32; unit < blocks * pairs; unit += kThreads / 32) {
    const int pair = unit / blocks, i = (unit - pair * blocks) * 32 + lane;
    if (i >= touched) continue;
    const int e = s.list[i], t = c0 + e, row0 = first_row + 2 * pair;
    T z[2];
    bool keep[2];
#pragma unroll
    for (int r = 0; r < 2; r++) {
      keep[r] = row0 + r < last_row;
      if (!keep[r]) continue;
      z[r] = in0[(row0 + r) * P.row_stride + t];
      if (P.allowed) keep[r] = mask_of(row0 + r)[t >> 5] >> (t & 31) & 1;
    }
    const uint32_t w = s.count[e];
    float bias = 0.0f;
    if (w & kBiased)
      for (int j = 0; j < s.num_biased; j++)
        if (s.biased[j] == e) bias = s.bias[j];
#pragma unroll
    for (int r = 0; r < 2; r++) {
      if (!keep[r]) continue;
      uint32_t count = w & kCount;
      if (w & kDrafted) {
        // the root (node 0) is the text's last token already
        const uint64_t path = s.path[row0 + r];
        for (int j = 1; j <= row0 + r; j++) count += s.drafted[j] == e && (path >> j & 1);
      }
      float x = E::load(z[r]);
      if (count || (w & kInPrompt)) x = x > 0.0f ? x / rho : x * rho;
      if (count) x = fmaf(-freq, static_cast<float>(count), x) - pres;
      if (w & kBiased) x += bias;
      out0[(row0 + r) * P.out_row_stride + t] = E::store(x);
    }
  }
}

template <int kChunk, int kThreads> int smem_of(const Params& P) {
  const int most = P.L + P.R + P.num_bias;
  return static_cast<int>(sizeof(Text<kChunk, kThreads / 32>)) + 2 * (most < kChunk ? most : kChunk);
}

template <int DT, int kChunk, int kThreads, Layout kLayout>
cudaError_t run(const Params& P, int B, cudaStream_t stream) {
  const int smem = smem_of<kChunk, kThreads>(P);
  // The most that any call takes, not this one's: the limit is the function's, and another
  // thread may launch it between these two calls.
  constexpr int kMost = static_cast<int>(sizeof(Text<kChunk, kThreads / 32>)) + 2 * kChunk;
  if (kMost > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(logits_kernel<DT, kChunk, kThreads, kLayout>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
  }
  const dim3 grid((P.V + kChunk - 1) / kChunk, B, (P.R + P.rows - 1) / P.rows);
  logits_kernel<DT, kChunk, kThreads, kLayout><<<grid, kThreads, smem, stream>>>(P);
  return cudaSuccess;
}

template <int DT, Layout kLayout>
cudaError_t launch(Params& P, int B, cudaStream_t stream) {
  P.rows = P.R < kMaxRows ? P.R : kMaxRows;
  // Large chunks read the text less often; small ones fill the machine where
  // requests are few: from half as many chunks of 8192 as SMs on, those (32 nodes: 4
  // requests 20.0 us with 1024 and 19.7 with 8192 entries, 8 requests 37.3 and 27.5;
  // two rows: 4 requests 7.6 and 8.3, 6 requests 10.3 and 6.3).
  const int64_t chunks = static_cast<int64_t>(B) * ((P.V + 8191) / 8192);
  if (chunks < kSms / 2) return run<DT, 1024, 256, kLayout>(P, B, stream);
  // With few rows a block's text outweighs them, and chunks of twice the size halve it
  // (512 requests of two rows 94 us, 132 with 8192; 64 chains of five 41.5 and 43.9; but
  // 16 requests of five 20.6 and 19.0, 32 nodes 78 and 74).
  static_assert(sizeof(Text<16384, 16>) + 2 * 16384 <= 113 * 1024, "two blocks to an SM");
  if (chunks >= 3 * kSms && P.rows < 7)
    return run<DT, 16384, 512, kLayout>(P, B, stream);
  return run<DT, 8192, 512, kLayout>(P, B, stream);
}

template <int DT> cudaError_t launch(Params& P, int B, Layout layout, cudaStream_t stream) {
  switch (layout) {
    case kAligned: return launch<DT, kAligned>(P, B, stream);
    case kShifted: return launch<DT, kShifted>(P, B, stream);
    default: return launch<DT, kSingle>(P, B, stream);
  }
}

}  // namespace

extern "C" {

specv_status spec_process_logits(const void* logits, int64_t batch_stride, int64_t row_stride,
                                 specv_dtype dtype, int B, int R, int V, const int32_t* tokens,
                                 const int32_t* parents, const int32_t* n_rows,
                                 const int32_t* history, int64_t history_stride, int L,
                                 const int32_t* seq_lens, const int32_t* prompt_lens,
                                 const float* repetition, const float* frequency,
                                 const float* presence, const int32_t* bias_tokens,
                                 const float* bias_values, int num_bias, const int32_t* allowed,
                                 void* out, int64_t out_batch_stride, int64_t out_row_stride,
                                 int32_t* status, specv_stream_t stream) {
  if (dtype != SPECV_F32 && dtype != SPECV_BF16) return SPECV_ERR_INVALID_ARG;
  if (!logits || !out || (L > 0 && !history) || !seq_lens || !status || (R > 1 && !tokens) || B < 1 || R < 1 ||
      V < 1 || L < 0 || num_bias < 0 || (num_bias > 0 && (!bias_tokens || !bias_values)))
    return SPECV_ERR_INVALID_ARG;
  const size_t size = dtype == SPECV_F32 ? 4 : 2;
  if (!aligned_to(logits, size) || !aligned_to(out, size)) return SPECV_ERR_INVALID_ARG;
  const void* words[] = {tokens,    parents,     n_rows,      history, seq_lens, prompt_lens, repetition,
                         frequency, presence,    bias_tokens, bias_values, allowed, status};
  for (const void* p : words)
    if (!aligned_to(p, 4)) return SPECV_ERR_INVALID_ARG;
  if (batch_stride < 0 || row_stride < 0 || out_batch_stride < 0 || out_row_stride < 0 || history_stride < 0)
    return SPECV_ERR_INVALID_ARG;
  if (logits == out && (batch_stride != out_batch_stride || row_stride != out_row_stride))
    return SPECV_ERR_INVALID_ARG;
  if (B > SPECV_MAX_BATCH || R > SPECV_MAX_NODES || V > specv_max_vocab(dtype) ||
      num_bias > SPECV_MAX_BIAS || L > (1 << 28))
    return SPECV_ERR_UNSUPPORTED;
  Params P{static_cast<const char*>(logits),
                 static_cast<char*>(out),
                 batch_stride,
                 row_stride,
                 out_batch_stride,
                 out_row_stride,
                 tokens,
                 parents,
                 n_rows,
                 history,
                 history_stride,
                 seq_lens,
                 prompt_lens,
                 repetition,
                 frequency,
                 presence,
                 bias_tokens,
                 bias_values,
                 allowed,
                 status,
                 R,
                 V,
                 L,
                 num_bias,
                 R};
  const int64_t n = static_cast<int64_t>(size);
  const bool alike = (reinterpret_cast<uintptr_t>(logits) - reinterpret_cast<uintptr_t>(out)) % 16 == 0 &&
                     (batch_stride - out_batch_stride) * n % 16 == 0 &&
                     (row_stride - out_row_stride) * n % 16 == 0;
  const bool aligned = aligned_to(logits, 16) && batch_stride * n % 16 == 0 && row_stride * n % 16 == 0;
  const Layout layout = !alike ? kSingle : aligned ? kAligned : kShifted;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == SPECV_F32 ? launch<SPECV_F32>(P, B, layout, st)
                                           : launch<SPECV_BF16>(P, B, layout, st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return SPECV_ERR_CUDA;
  }
  return launched();
}

}  // extern "C"
