// The prompt's pass over the paged cache, host side of its attention.

#include "chunk.cuh"

using namespace specv_chunk;

namespace specv_chunk {

template <> cudaError_t run<Bf16>(const Params&, const CUtensorMap&, const CUtensorMap&, cudaStream_t);
template <> cudaError_t run<F16>(const Params&, const CUtensorMap&, const CUtensorMap&, cudaStream_t);

}  // namespace specv_chunk

namespace {

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// The workspace for calls of up to `longest` tokens a request.
struct Plan {
  int part_rows;
  size_t stats, parts, total;  // offsets; before them the cuts

  Plan(int longest, int group, int head_dim) {
    const int64_t rows = static_cast<int64_t>(longest) * group;
    const int dim = head_dim <= 64 ? 64 : 128;
    part_rows = static_cast<int>(rows < kRowTile ? rows : kRowTile) + 7 & ~7;
    stats = align256(kMaxCtas * sizeof(Cut));
    parts = stats + align256(2 * kMaxCtas * part_rows * sizeof(float2));
    total = parts + align256(2 * kMaxCtas * part_rows * dim * sizeof(float));
  }
};

// Rows of one request are counted in 32 bits.
bool too_long(int longest, int group) { return static_cast<int64_t>(longest) * group > INT_MAX / 4; }

}  // namespace

extern "C" {

size_t specv_chunk_workspace_bytes(int longest, int q_heads, int kv_heads, int head_dim) {
  if (longest < 1 || kv_heads < 1 || q_heads < kv_heads || q_heads > 1024 || q_heads % kv_heads != 0 ||
      head_dim < 8 || head_dim > SPECV_MAX_HEAD_DIM || head_dim % 8 != 0 ||
      too_long(longest, q_heads / kv_heads))
    return 0;
  return Plan(longest, q_heads / kv_heads, head_dim).total;
}

specv_status spec_chunk_attention(const specv_cache* cache, const specv_rows* q,
                                  const int32_t* cu_tokens, int B, int T, int longest, int q_heads,
                                  float scale, float cap, int window, const int32_t* prefix_lens,
                                  const float* slopes, const specv_rows* out, int32_t* status,
                                  void* workspace, size_t workspace_bytes, specv_stream_t stream) {
  const specv_status s = check_cache(cache, B, 1);
  if (s != SPECV_OK) return s;
  if (!rows_ok(q) || !rows_ok(out) || !cu_tokens || !status || !workspace || cache->layers != 1 ||
      T < 0 || longest < 1 || q_heads < 1 || q_heads % cache->heads != 0 || !(scale > 0.0f) ||
      scale > 1e30f || !(cap >= 0.0f) || cap > 1e30f || window < 0)
    return SPECV_ERR_INVALID_ARG;
  if (!aligned_to(cu_tokens, 4) || !aligned_to(prefix_lens, 4) || !aligned_to(slopes, 4) ||
      !aligned_to(status, 4) || !aligned_to(workspace, 256))
    return SPECV_ERR_INVALID_ARG;
  const int group = q_heads / cache->heads;
  if (q_heads > 1024 || B > kMaxRequests || too_long(longest, group)) return SPECV_ERR_UNSUPPORTED;
  // the scores' factor in the cap's tanh, a 32-bit number as what follows from it is
  const double unit = cap > 0.0f ? static_cast<double>(scale) / cap : 0.0, turn = 2.0 * unit * 1.4426950408889634;
  if (turn > 1e30 || (cap > 0.0f && turn < 1e-30)) return SPECV_ERR_INVALID_ARG;
  const Plan plan(longest, group, cache->head_dim);
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
  // Tensor copies, the largest that fit pages and tiles alike, from 16 rows on.
  const int page = cache->page_size, fit = page & -page;
  int box_rows = fit < 16 ? 0 : fit < kKeys ? fit : kKeys;
  CUtensorMap k_map = {}, v_map = {};
  if (box_rows && (!tensor_map(&k_map, cache, cache->k, box_rows) ||
                   !tensor_map(&v_map, cache, cache->v, box_rows)))
    box_rows = 0;
  // cap tanh(z) in units of log 2 as z * poly(z^2), for |z| <= 0.6 (chunk.cuh).
  static const double kTanh[5] = {0.9999999268676429, -0.33332309962801215, 0.13310173497792807,
                                  -0.05210147302447307, 0.015475417666045245};
  float poly[5];
  for (int i = 0; i < 5; i++) poly[i] = static_cast<float>(kTanh[i] * cap * 1.4426950408889634);
  const float small = cap > 0.0f ? static_cast<float>(0.6 / unit) : 0.0f;
  const Params P{to_cache(cache),
                 to_rows(q),
                 to_rows(out),
                 ws,
                 cu_tokens,
                 prefix_lens,
                 slopes,
                 status,
                 B,
                 T,
                 longest,
                 q_heads,
                 group,
                 window ? window : INT_MAX,
                 ctas,
                 plan.part_rows,
                 box_rows,
                 scale * 1.4426950408889634f,
                 cap * 1.4426950408889634f,
                 static_cast<float>(unit),
                 small,
                 {poly[0], poly[1], poly[2], poly[3], poly[4]}};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->dtype == SPECV_BF16 ? run<Bf16>(P, k_map, v_map, st)
                                                   : run<F16>(P, k_map, v_map, st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return SPECV_ERR_CUDA;
  }
  return SPECV_OK;
}

}  // extern "C"
