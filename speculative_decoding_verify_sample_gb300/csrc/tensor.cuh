// The tensor cores, tensor memory, barriers and copies as the attention kernels use
// them: thin wrappers of the instructions, and the waits, which all end.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "cache.cuh"

namespace specv_tensor {

// How long a wait lasts before it gives up.  (A build with less than a millisecond polls:
// try_wait itself may last longer.  With 0 it gives up wherever it would wait.)
#ifndef SPECV_ATTENTION_WAIT_NS
#define SPECV_ATTENTION_WAIT_NS 2000000000ull
#endif
constexpr uint64_t kWaitNs = SPECV_ATTENTION_WAIT_NS;
constexpr bool kPolls = kWaitNs < 1000000;

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

__device__ __forceinline__ bool barrier_test(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
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

// Waits for a phase, two seconds at most: then, and from then on in the whole CTA,
// no wait lasts any more.  False if the phase is not over: who waited for it leaves its
// loop and arrives nowhere, so that no other takes a copy or an MMA for done that is not.
__device__ __forceinline__ bool barrier_wait_slow(uint32_t bar, uint32_t parity, volatile int* gave_up) {
  const uint64_t start = now_ns();
  while (!(kPolls ? barrier_test(bar, parity) : barrier_try(bar, parity))) {
    if (*gave_up) return false;
    if (now_ns() - start >= kWaitNs) {
      *gave_up = 1;
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ bool barrier_wait(uint32_t bar, uint32_t parity, volatile int* gave_up) {
  return (!kPolls && barrier_try(bar, parity)) || barrier_wait_slow(bar, parity, gave_up);
}

// Waits for this thread's own work in flight, a second at most, whatever gave up.
__device__ __forceinline__ void barrier_wait_own(uint32_t bar, uint32_t parity) {
  const uint64_t start = now_ns();
  while (!barrier_try(bar, parity) && now_ns() - start < 1000000000ull) {
  }
}

__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from),
               "r"(real ? 16 : 0)
               : "memory");
}

__device__ __forceinline__ void barrier_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void tensor_copy(uint32_t to, const CUtensorMap* map, int d, int row,
                                            int head, int page, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(to),
      "l"(map), "r"(d), "r"(row), "r"(head), "r"(page), "r"(bar)
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

// 64 columns, waited for.
__device__ __forceinline__ void tmem_load64(uint32_t at, uint32_t (&x)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : SPECV_R32(x, 0), SPECV_R32(x, 32)
      : "r"(at), "r"(at + 32)
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

__device__ __forceinline__ void tmem_store32(uint32_t at, const uint32_t (&x)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::SPECV_I8(x, 0),
      SPECV_I8(x, 8), SPECV_I8(x, 16), SPECV_I8(x, 24), "r"(at)
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

// Whether it holds for one of the 256 threads of the softmax, which wait for one another.
__device__ __forceinline__ bool any_of_softmax(bool x) {
  uint32_t any;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
      " barrier.cta.red.or.pred q, 1, 256, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(any)
      : "r"(static_cast<uint32_t>(x))
      : "memory");
  return any;
}

__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Host side ---------------------------------------------------------------

// The tensor map of a cache: [page, head, row, d], boxes of 64 columns and
// box_rows rows of a page, a multiple of eight as the swizzled groups are.
inline bool tensor_map(CUtensorMap* map, const specv_cache* c, void* data, int box_rows) {
  using Encode = decltype(&cuTensorMapEncodeTiled);
  static const Encode encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<Encode>(fn);
  }();
  if (!encode) return false;
  const int64_t row = static_cast<int64_t>(c->head_dim) * 2;
  const cuuint64_t size[4] = {static_cast<cuuint64_t>(c->head_dim), static_cast<cuuint64_t>(c->page_size),
                              static_cast<cuuint64_t>(c->heads), static_cast<cuuint64_t>(c->pages)};
  const int64_t bytes[3] = {c->row_stride * 2, c->head_stride * 2, c->page_stride * 2};
  cuuint64_t stride[3];
  for (int i = 0; i < 3; i++) {
    if (size[i + 1] > 1 && (bytes[i] < row || bytes[i] >= 1ll << 40)) return false;
    stride[i] = size[i + 1] > 1 ? static_cast<cuuint64_t>(bytes[i]) : static_cast<cuuint64_t>(row);
  }
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_rows), 1, 1}, step[4] = {1, 1, 1, 1};
  return encode(map, c->dtype == SPECV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                            : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                4, data, size, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace specv_tensor
