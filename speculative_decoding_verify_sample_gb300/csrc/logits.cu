// Penalties for repeated tokens, biases and grammar masks on the logits of a
// drafted tree's (or chain's) rows.

#include "cache.cuh"

using namespace specv_cache_ops;

namespace {

constexpr int kThreads = 256;
constexpr int kInFlight = 4;  // vectors a thread has in flight

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

// A block takes kChunk vocabulary entries of one request, for all its rows:
// it counts the text's tokens among them once, in shared memory, and streams
// the rows through.  kVec elements go at a time (16 bytes; 1 where the input
// and the output are not aligned alike).
template <int DT, int kChunk, int kVec>
__global__ void __launch_bounds__(kThreads) logits_kernel(const Params P) {
  using E = Elt<DT>;
  using T = typename E::T;
  struct __align__(kVec * sizeof(T)) Vec {
    T x[kVec];
  };
  __shared__ uint32_t s_count[kChunk];
  __shared__ float s_bias[kChunk];
  __shared__ uint32_t s_touched[kChunk / 32 + 1];
  __shared__ uint64_t s_path[kMaxNodes];
  __shared__ int s_drafted[kMaxNodes];  // chunk entry of node i's token, -1 where it is another's
  __shared__ int s_n, s_bad;

  const int tid = threadIdx.x, lane = tid & 31, b = blockIdx.y;
  const int c0 = blockIdx.x * kChunk, c1 = min(P.V, c0 + kChunk);
  for (int e = tid; e < kChunk; e += kThreads) s_count[e] = 0;
  for (int e = tid; e < kChunk / 32 + 1; e += kThreads) s_touched[e] = 0;

  const int total = P.seq_lens[b], prompt = P.prompt_lens ? P.prompt_lens[b] : 0;
  const float rho = P.repetition ? P.repetition[b] : 1.0f;
  const float freq = P.frequency ? P.frequency[b] : 0.0f;
  const float pres = P.presence ? P.presence[b] : 0.0f;
  if (tid < 32) {
    Tree t = read_tree(P.parents, P.n_rows, P.seq_lens, b, P.R, INT64_MAX, lane);
    bool bad_token = false;
    if (!(t.bad & SPECV_DEV_BAD_TREE)) {
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
        s_drafted[i] = at;
      }
      uint64_t bits[2];
      ancestors(t, lane, bits);
      s_path[lane] = bits[0];
      s_path[lane + 32] = bits[1];
    }
    if (__any_sync(kFullMask, bad_token)) t.bad |= SPECV_DEV_BAD_TOKEN;
    if (total > P.L || prompt < 0 || prompt > total) t.bad |= SPECV_DEV_BAD_CACHE;
    if (!(rho > 0.0f) || !isfinite(rho) || !isfinite(freq) || !isfinite(pres))
      t.bad |= SPECV_DEV_BAD_PENALTY;
    if (lane == 0) {
      s_n = t.n;
      s_bad = static_cast<int>(t.bad);
    }
  }
  __syncthreads();

  // The text's tokens in this chunk.  Counts are whole numbers: the order in
  // which the threads add does not show.
  bool bad_token = false;
  if (!s_bad) {
    const int32_t* hist = P.history + b * P.history_stride;
    for (int i = tid; i < total; i += kThreads) {
      const int token = hist[i];
      bad_token |= token < 0 || token >= P.V;
      if (token >= c0 && token < c1) {
        if (i < prompt) atomicOr(&s_count[token - c0], kInPrompt);
        else atomicAdd(&s_count[token - c0], 1u);
        atomicOr(&s_touched[(token - c0) / 32], 1u << ((token - c0) & 31));
      }
    }
    if (tid < s_n && s_drafted[tid] >= 0) {
      const int e = s_drafted[tid];
      atomicOr(&s_count[e], kDrafted);
      atomicOr(&s_touched[e / 32], 1u << (e & 31));
    }
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
        s_bias[token - c0] = sum;
        atomicOr(&s_count[token - c0], kBiased);
        atomicOr(&s_touched[(token - c0) / 32], 1u << ((token - c0) & 31));
      }
    }
  }
  const bool any_bad = __syncthreads_or(bad_token);
  const int bad = s_bad | (any_bad ? SPECV_DEV_BAD_TOKEN : 0);
  if (blockIdx.x == 0 && tid == 0) P.status[b] = bad;
  const int n = s_n ? s_n : P.R;

  auto changed = [&](float z, int e, int row) {
    const uint32_t word = s_count[e];
    uint32_t count = word & kCount;
    if (word & kDrafted) {
      // the root (node 0) is the text's last token already
      const uint64_t path = s_path[row];
      for (int j = 1; j <= row; j++) count += s_drafted[j] == e && (path >> j & 1);
    }
    if (count || (word & kInPrompt)) z = z > 0.0f ? z / rho : z * rho;
    if (count) z = fmaf(-freq, static_cast<float>(count), z) - pres;
    if (word & kBiased) z += s_bias[e];
    return z;
  };

  constexpr int kVecs = kChunk / kVec + (kVec > 1);  // one more where a row starts inside a vector
  const int64_t words = (P.V + 31) / 32;
  for (int w0 = tid; w0 < n * kVecs; w0 += kThreads * kInFlight) {
    Vec data[kInFlight];
    uint32_t keep[kInFlight];
    int row[kInFlight], at[kInFlight];  // a vector's row and first entry; may begin before c0
#pragma unroll
    for (int u = 0; u < kInFlight; u++) {
      const int w = w0 + u * kThreads;
      row[u] = w / kVecs;
      at[u] = c1;
      keep[u] = 0;
      if (w >= n * kVecs) continue;
      const T* in = reinterpret_cast<const T*>(P.in) + b * P.batch_stride + row[u] * P.row_stride;
      const int lead =
          kVec == 1 ? 0
                    : static_cast<int>(reinterpret_cast<uintptr_t>(in + c0) / sizeof(T) % kVec);
      at[u] = c0 - lead + (w - row[u] * kVecs) * kVec;
      if (at[u] >= c1 || bad) continue;
      keep[u] = (1u << kVec) - 1;
      const int from = max(at[u], c0), to = min(at[u] + kVec, c1);
      if (P.allowed) {
        const int32_t* bits = P.allowed + (static_cast<int64_t>(b) * P.R + row[u]) * words;
        uint64_t both = static_cast<uint32_t>(bits[from >> 5]);
        if ((to - 1) >> 5 != from >> 5) both |= static_cast<uint64_t>(bits[(to - 1) >> 5]) << 32;
        keep[u] &= static_cast<uint32_t>(both >> (from & 31)) << (from - at[u]);
      }
      if (keep[u] == 0) continue;
      if (from == at[u] && to == at[u] + kVec) {
        data[u] = *reinterpret_cast<const Vec*>(in + at[u]);
      } else {
#pragma unroll
        for (int e = 0; e < kVec; e++)
          if (at[u] + e >= from && at[u] + e < to) data[u].x[e] = in[at[u] + e];
      }
    }
#pragma unroll
    for (int u = 0; u < kInFlight; u++) {
      if (at[u] >= c1) continue;
      const int from = max(at[u], c0), to = min(at[u] + kVec, c1);
      uint64_t window = 0;  // touched bits from `from` on
      if (!bad) {
        const int e = from - c0;
        window = (static_cast<uint64_t>(s_touched[e / 32 + 1]) << 32 | s_touched[e / 32]) >> (e & 31);
      }
      const uint32_t touched = static_cast<uint32_t>(window) << (from - at[u]) & keep[u];
#pragma unroll
      for (int e = 0; e < kVec; e++)
        if (!(keep[u] >> e & 1)) data[u].x[e] = E::kNegInf;
      if (touched) {
#pragma unroll
        for (int e = 0; e < kVec; e++)
          if ((touched >> e & 1) && at[u] + e < c1)
            data[u].x[e] = E::store(changed(E::load(data[u].x[e]), at[u] + e - c0, row[u]));
      }
      T* out = reinterpret_cast<T*>(P.out) + b * P.out_batch_stride + row[u] * P.out_row_stride;
      if (from == at[u] && to == at[u] + kVec) {
        *reinterpret_cast<Vec*>(out + at[u]) = data[u];
      } else {
#pragma unroll
        for (int e = 0; e < kVec; e++)
          if (at[u] + e >= from && at[u] + e < to) out[at[u] + e] = data[u].x[e];
      }
    }
  }
}

template <int DT, int kChunk>
specv_status launch(const Params& P, int B, bool vectors, cudaStream_t stream) {
  const dim3 grid((P.V + kChunk - 1) / kChunk, B);
  if (vectors) logits_kernel<DT, kChunk, DT == SPECV_F32 ? 4 : 8><<<grid, kThreads, 0, stream>>>(P);
  else logits_kernel<DT, kChunk, 1><<<grid, kThreads, 0, stream>>>(P);
  return launched();
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
  if (logits == out && (batch_stride != out_batch_stride || row_stride != out_row_stride))
    return SPECV_ERR_INVALID_ARG;
  if (B > SPECV_MAX_BATCH || R > SPECV_MAX_NODES || V > specv_max_vocab(dtype) ||
      num_bias > SPECV_MAX_BIAS || L > (1 << 28))
    return SPECV_ERR_UNSUPPORTED;
  const Params P{static_cast<const char*>(logits),
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
                 num_bias};
  const int64_t n = static_cast<int64_t>(size);
  const bool vectors = (reinterpret_cast<uintptr_t>(logits) - reinterpret_cast<uintptr_t>(out)) % 16 == 0 &&
                       (batch_stride - out_batch_stride) * n % 16 == 0 &&
                       (row_stride - out_row_stride) * n % 16 == 0;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return dtype == SPECV_F32 ? launch<SPECV_F32, 2048>(P, B, vectors, st)
                            : launch<SPECV_BF16, 2048>(P, B, vectors, st);
}

}  // extern "C"
