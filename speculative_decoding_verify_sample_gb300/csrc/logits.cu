// Penalties for repeated tokens, biases and grammar masks on the logits of a
// drafted tree's (or chain's) rows.

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
  int rows;     // of a block
  int shifted;  // rows do not all begin at a 16-byte boundary
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

// What a block needs of one request's text, for its chunk of the vocabulary.
template <int kChunk> struct Text {
  uint32_t count[kChunk];
  uint32_t touched[kChunk / 32];
  uint16_t list[kChunk];  // touched entries, each warp's from its first element on
  uint64_t path[kMaxNodes];
  float bias[SPECV_MAX_BIAS];      // sums of the biases in this chunk ...
  uint16_t biased[SPECV_MAX_BIAS]; // ... and their entries
  int drafted[kMaxNodes];  // entry of node i's token, -1 where it is another chunk's
  int num_biased, n, bad;
};

// A block takes kChunk vocabulary entries of one request, for P.rows of its
// rows.  It counts the text's tokens among them once, in shared memory, then
// streams the rows through: nearly every element is only masked and copied, 16
// bytes at a time (kVec elements; 1 where input and output are not aligned
// alike), and the few that the text, a draft or a bias touches are computed
// one to a lane and stored over the copy.  A warp owns the same columns in
// every row, so it alone orders the two stores; only where the rows' vectors
// are shifted against the chunk the block has to.
template <int DT, int kChunk, int kThreads, int kVec>
__global__ void __launch_bounds__(kThreads) logits_kernel(const Params P) {
  using E = Elt<DT>;
  using T = typename E::T;
  constexpr int kMine = kChunk / kVec / kThreads;         // vectors of a row a thread has
  constexpr int kBlock = kMine < 8 ? kMine : 8;           // ... in flight
  constexpr int kWords = kChunk / 32 / (kThreads / 32);   // bitmap words of a warp
  static_assert(kChunk % (kVec * kThreads) == 0 && kWords <= 32 && kWords % kMine == 0 || kVec == 1, "");
  struct __align__(kVec * sizeof(T)) Vec {
    T x[kVec];
  };
  extern __shared__ __align__(16) char smem[];
  Text<kChunk>& s = *reinterpret_cast<Text<kChunk>*>(smem);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, b = blockIdx.y;
  const int c0 = blockIdx.x * kChunk, c1 = min(P.V, c0 + kChunk);
  for (int e = tid; e < kChunk; e += kThreads) s.count[e] = 0;
  for (int e = tid; e < kChunk / 32; e += kThreads) s.touched[e] = 0;

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
        s.drafted[i] = at;
      }
      uint64_t bits[2];
      ancestors(t, lane, bits);
      s.path[lane] = bits[0];
      s.path[lane + 32] = bits[1];
    }
    if (__any_sync(kFullMask, bad_token)) t.bad |= SPECV_DEV_BAD_TOKEN;
    if (total > P.L || prompt < 0 || prompt > total) t.bad |= SPECV_DEV_BAD_CACHE;
    if (!(rho > 0.0f) || !isfinite(rho) || !isfinite(freq) || !isfinite(pres))
      t.bad |= SPECV_DEV_BAD_PENALTY;
    if (lane == 0) {
      s.n = t.n;
      s.bad = static_cast<int>(t.bad);
      s.num_biased = 0;
    }
  }
  __syncthreads();

  // The text's tokens in this chunk.  Counts are whole numbers: the order in
  // which the threads add does not show.
  bool bad_token = false;
  auto touch = [&](int e) { atomicOr(&s.touched[e / 32], 1u << (e & 31)); };
  if (!s.bad) {
    auto count = [&](int i, int token) {
      bad_token |= static_cast<unsigned>(token) >= static_cast<unsigned>(P.V);
      const int e = token - c0;
      if (e < 0 || token >= c1) return;
      if (i < prompt) atomicOr(&s.count[e], kInPrompt);
      else atomicAdd(&s.count[e], 1u);
      touch(e);
    };
    const int32_t* hist = P.history + b * P.history_stride;
    const int vectors = reinterpret_cast<uintptr_t>(hist) % 16 == 0 ? total / 4 : 0;
    for (int i = tid; i < vectors; i += kThreads) {
      const int4 t = reinterpret_cast<const int4*>(hist)[i];
      count(4 * i, t.x);
      count(4 * i + 1, t.y);
      count(4 * i + 2, t.z);
      count(4 * i + 3, t.w);
    }
    for (int i = 4 * vectors + tid; i < total; i += kThreads) count(i, hist[i]);
    if (tid < s.n && s.drafted[tid] >= 0) {
      atomicOr(&s.count[s.drafted[tid]], kDrafted);
      touch(s.drafted[tid]);
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
        const int at = atomicAdd(&s.num_biased, 1);
        s.biased[at] = static_cast<uint16_t>(token - c0);
        s.bias[at] = sum;
        atomicOr(&s.count[token - c0], kBiased);
        touch(token - c0);
      }
    }
  }
  const bool any_bad = __syncthreads_or(bad_token);
  const int bad = s.bad | (any_bad ? SPECV_DEV_BAD_TOKEN : 0);
  if (blockIdx.x == 0 && blockIdx.z == 0 && tid == 0) P.status[b] = bad;

  // This warp's touched entries: a bitmap word to a lane.  Its elements are
  // 32 kVec in a row, once in every kThreads kVec (kVec = 1: any share will do,
  // the block orders the stores).
  const int word = lane >= kWords ? 0
                   : kVec == 1    ? warp * kWords + lane
                                  : (lane / kVec * (kThreads / 32) + warp) * kVec + lane % kVec;
  uint32_t bits = lane < kWords && !bad ? s.touched[word] : 0;
  int upto = __popc(bits);
  const int own = upto;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int x = __shfl_up_sync(kFullMask, upto, o);
    if (lane >= o) upto += x;
  }
  const int fixes = __shfl_sync(kFullMask, upto, 31);
  uint16_t* list = s.list + warp * kWords * 32;
  for (int at = upto - own; bits; bits &= bits - 1)
    list[at++] = static_cast<uint16_t>(word * 32 + __ffs(bits) - 1);
  __syncwarp();

  auto changed = [&](float z, int e, int row) {
    const uint32_t w = s.count[e];
    uint32_t count = w & kCount;
    if (w & kDrafted) {
      // the root (node 0) is the text's last token already
      const uint64_t path = s.path[row];
      for (int j = 1; j <= row; j++) count += s.drafted[j] == e && (path >> j & 1);
    }
    if (count || (w & kInPrompt)) z = z > 0.0f ? z / rho : z * rho;
    if (count) z = fmaf(-freq, static_cast<float>(count), z) - pres;
    if (w & kBiased)
      for (int j = 0; j < s.num_biased; j++)
        if (s.biased[j] == e) z += s.bias[j];
    return z;
  };

  const int n = s.n ? s.n : P.R;
  const int first_row = blockIdx.z * P.rows, last_row = min(n, first_row + P.rows);
  const int64_t words = (P.V + 31) / 32;
  for (int row = first_row; row < last_row; row++) {
    const T* in = reinterpret_cast<const T*>(P.in) + b * P.batch_stride + row * P.row_stride;
    T* out = reinterpret_cast<T*>(P.out) + b * P.out_batch_stride + row * P.out_row_stride;
    const int32_t* mask =
        P.allowed ? P.allowed + (static_cast<int64_t>(b) * P.R + row) * words : nullptr;
    const int lead =
        kVec == 1 || !P.shifted
            ? 0
            : static_cast<int>(reinterpret_cast<uintptr_t>(in + c0) / sizeof(T) % kVec);
    auto allowed = [&](int t) { return !mask || (mask[t >> 5] >> (t & 31) & 1); };
    // the first of the touched elements, in flight with the copies
    T fix = 0;
    int fix_at = lane < fixes ? list[lane] : -1;
    if (fix_at >= 0 && !allowed(c0 + fix_at)) fix_at = -1;
    if (fix_at >= 0) fix = in[c0 + fix_at];
#pragma unroll 1
    for (int u0 = 0; u0 < kMine; u0 += kBlock) {
      Vec data[kBlock];
      uint32_t keep[kBlock];
#pragma unroll
      for (int u = 0; u < kBlock; u++) {
        const int at = c0 - lead + ((u0 + u) * kThreads + tid) * kVec;
        const int from = max(at, c0), to = min(at + kVec, c1);
        keep[u] = 0;
        if (from < to && !bad) {
          keep[u] = (1u << kVec) - 1;
          if (mask) {
            uint64_t both = static_cast<uint32_t>(mask[from >> 5]);
            if ((to - 1) >> 5 != from >> 5) both |= static_cast<uint64_t>(mask[(to - 1) >> 5]) << 32;
            keep[u] &= static_cast<uint32_t>(both >> (from & 31)) << (from - at);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kBlock; u++) {
        const int at = c0 - lead + ((u0 + u) * kThreads + tid) * kVec;
        if (keep[u] == 0) continue;  // nothing to read
        if (at >= c0 && at + kVec <= c1) {
          data[u] = *reinterpret_cast<const Vec*>(in + at);
        } else {
#pragma unroll
          for (int e = 0; e < kVec; e++)
            if (at + e >= c0 && at + e < c1) data[u].x[e] = in[at + e];
        }
      }
#pragma unroll
      for (int u = 0; u < kBlock; u++) {
        const int at = c0 - lead + ((u0 + u) * kThreads + tid) * kVec;
#pragma unroll
        for (int e = 0; e < kVec; e++)
          if (!(keep[u] >> e & 1)) data[u].x[e] = E::kNegInf;
        if (at >= c0 && at + kVec <= c1) {
          *reinterpret_cast<Vec*>(out + at) = data[u];
        } else {
#pragma unroll
          for (int e = 0; e < kVec; e++)
            if (at + e >= c0 && at + e < c1) out[at + e] = data[u].x[e];
        }
      }
    }
    if (lead && tid < lead) {  // what the shifted vectors leave at the chunk's end
      const int t = c0 + kChunk - lead + tid;
      if (t < c1) out[t] = bad || !allowed(t) ? static_cast<T>(E::kNegInf) : in[t];
    }
    if (kVec == 1 || P.shifted) __syncthreads();
    else __syncwarp();
    if (fix_at >= 0) out[c0 + fix_at] = E::store(changed(E::load(fix), fix_at, row));
    for (int i = lane + 32; i < fixes; i += 32) {
      const int e = list[i];
      if (allowed(c0 + e)) out[c0 + e] = E::store(changed(E::load(in[c0 + e]), e, row));
    }
  }
}

template <int DT, int kChunk, int kThreads, int kVec>
cudaError_t run(const Params& P, int B, cudaStream_t stream) {
  constexpr int kSmem = sizeof(Text<kChunk>);
  if (kSmem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(logits_kernel<DT, kChunk, kThreads, kVec>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
  }
  const dim3 grid((P.V + kChunk - 1) / kChunk, B, (P.R + P.rows - 1) / P.rows);
  logits_kernel<DT, kChunk, kThreads, kVec><<<grid, kThreads, kSmem, stream>>>(P);
  return cudaSuccess;
}

// Large chunks read the text less often; small ones fill the machine where
// requests are few.
template <int DT>
cudaError_t launch(Params& P, int B, bool vectors, cudaStream_t stream) {
  constexpr int kVec = DT == SPECV_F32 ? 4 : 8;
  if (static_cast<int64_t>(B) * ((P.V + 8191) / 8192) >= 304) {
    P.rows = P.R;
    return vectors ? run<DT, 8192, 256, kVec>(P, B, stream) : run<DT, 8192, 256, 1>(P, B, stream);
  }
  P.rows = P.R < 8 ? P.R : 8;
  return vectors ? run<DT, 1024, 128, kVec>(P, B, stream) : run<DT, 1024, 128, 1>(P, B, stream);
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
                 R,
                 0};
  // A row's place against 16 bytes: the same in the output, or single elements go.
  const int64_t n = static_cast<int64_t>(size);
  const bool vectors = (reinterpret_cast<uintptr_t>(logits) - reinterpret_cast<uintptr_t>(out)) % 16 == 0 &&
                       (batch_stride - out_batch_stride) * n % 16 == 0 &&
                       (row_stride - out_row_stride) * n % 16 == 0;
  P.shifted = reinterpret_cast<uintptr_t>(logits) % 16 != 0 || batch_stride * n % 16 != 0 ||
              row_stride * n % 16 != 0;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == SPECV_F32 ? launch<SPECV_F32>(P, B, vectors, st)
                                           : launch<SPECV_BF16>(P, B, vectors, st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return SPECV_ERR_CUDA;
  }
  return launched();
}

}  // extern "C"
