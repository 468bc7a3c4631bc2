// What the kernels on the tensor cores share: mbarriers with bounded waits, asynchronous copies,
// tcgen05 products and TMEM accesses, and conversions.  Device code only.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

namespace ula_tc {

// Copies the count of ula_rows_score's warps whose waits ran out, in all launches so far (ula_score.cu).
__attribute__((visibility("hidden"))) cudaError_t score_late(uint32_t *late, cudaStream_t st);

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Bounded: false after 2^18 tries. A try that is not met comes back after 4.0 us on this GPU,
// whatever time it is given, so a wait that is never met ends after 1.05 s, and any wait that these
// kernels can meet is shorter than a tenth of a millisecond.  (Waiting for the kernel before has no limit of
// theirs and comes first.) The loop is written out because its
// size matters: the compute warps pass through some 15 waits a tile, their code is longer than
// the instruction caches nearest to them: with a clock read and two ways out in each wait the step
// of 96 tokens, 128 heads, 2,051 rows took 6 % more when this form came in, and with a limit that is
// a kernel argument it takes 125.0 us instead of 120.5.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n .reg .u32 i;\n mov.u32 i, 0;\n"
      "again:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra over;\n"
      " add.u32 i, i, 1;\n setp.lt.u32 p, i, 0x40000;\n @p bra again;\n setp.ne.u32 p, 0, 0;\n"
      "over:\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done) : "r"(bar), "r"(parity) : "memory");
  return done;
}

// By a whole warp: the same answer in every lane, so that a warp leaves its work as one.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

// Two or three phases, asked for together: an answer takes 150 to 250 clocks when shared memory is busy, and the
// answers to one after the other as many times that.  (A round of tries that are not met takes as much
// longer, so there are fewer of them.)
__device__ __forceinline__ bool warp_wait(uint32_t bar0, uint32_t parity0, uint32_t bar1, uint32_t parity1) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .u32 i;\n mov.u32 i, 0;\n"
      "again:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n and.pred p, p, q;\n @p bra over;\n"
      " add.u32 i, i, 1;\n setp.lt.u32 p, i, 0x20000;\n @p bra again;\n setp.ne.u32 p, 0, 0;\n"
      "over:\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done) : "r"(bar0), "r"(parity0), "r"(bar1), "r"(parity1) : "memory");
  return __all_sync(0xffffffffu, done);
}
__device__ __forceinline__ bool warp_wait(uint32_t bar0, uint32_t parity0, uint32_t bar1, uint32_t parity1, uint32_t bar2, uint32_t parity2) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p, q, r;\n .reg .u32 i;\n mov.u32 i, 0;\n"
      "again:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n mbarrier.try_wait.parity.shared::cta.b64 r, [%5], %6;\n"
      " and.pred p, p, q;\n and.pred p, p, r;\n @p bra over;\n"
      " add.u32 i, i, 1;\n setp.lt.u32 p, i, 0x15555;\n @p bra again;\n setp.ne.u32 p, 0, 0;\n"
      "over:\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done) : "r"(bar0), "r"(parity0), "r"(bar1), "r"(parity1), "r"(bar2), "r"(parity2) : "memory");
  return __all_sync(0xffffffffu, done);
}

// Whether a phase has ended, asked without waiting: the answer takes some 250 clocks when shared memory is
// busy, in which the warp goes on with what does not need it.
__device__ __forceinline__ uint32_t mbar_ended(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(done) : "r"(bar), "r"(parity) : "memory");
  return done;
}

// The same of two, asked together.
__device__ __forceinline__ uint32_t mbar_ended(uint32_t bar0, uint32_t parity0, uint32_t bar1, uint32_t parity1) {
  uint32_t done;
  asm volatile("{\n .reg .pred p, q;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
               " mbarrier.test_wait.parity.shared::cta.b64 q, [%3], %4;\n and.pred p, p, q;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(done) : "r"(bar0), "r"(parity0), "r"(bar1), "r"(parity1) : "memory");
  return done;
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p;
}

// One MMA of K = 16: D[128][N] (+)= A B, all operands in shared memory (bf16, or f16 as idesc says).
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc) : "memory");
}

// The same with A in TMEM: row i in lane i, two elements of K in a column.
__device__ __forceinline__ void mma_tmem_a(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc) : "memory");
}

// 16 lanes of TMEM by 8 columns: thread t gives lane t / 4 columns 2 (t % 4) and the next, from v[0] and
// v[1], and lane t / 4 + 8 the same, from v[2] and v[3]; four times, 8 columns on.
__device__ __forceinline__ void tmem_st_16x32(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
      ::"r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(addr) : "memory");
}

// 16 bytes to shared memory without passing through registers; zeros where `bytes` is 0.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// This thread's arrival, once its copies so far have landed.
__device__ __forceinline__ void copy_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Brings bytes (a multiple of 16, as the address is) into L2.
__device__ __forceinline__ void prefetch(const void *src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// Bytes to shared memory (a multiple of 16, as both addresses are), counted by an mbarrier.
__device__ __forceinline__ void copy_bulk(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// N consecutive TMEM columns of this warp's 32 lanes.
template <int N> __device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[N]);
template <int N> __device__ __forceinline__ void tmem_st(uint32_t addr, const float (&v)[N]);
template <> __device__ __forceinline__ void tmem_ld<4>(uint32_t addr, float (&v)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(addr) : "memory");
}
template <> __device__ __forceinline__ void tmem_ld<8>(uint32_t addr, float (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
                 "=f"(v[7]) : "r"(addr) : "memory");
}
template <> __device__ __forceinline__ void tmem_ld<16>(uint32_t addr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]),
        "=f"(v[15]) : "r"(addr) : "memory");
}
template <> __device__ __forceinline__ void tmem_ld<32>(uint32_t addr, float (&v)[32]) {
  tmem_ld<16>(addr, reinterpret_cast<float (&)[16]>(v[0]));
  tmem_ld<16>(addr + 16, reinterpret_cast<float (&)[16]>(v[16]));
}
template <> __device__ __forceinline__ void tmem_st<4>(uint32_t addr, const float (&v)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%4], {%0, %1, %2, %3};"
               ::"f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "r"(addr) : "memory");
}

__device__ __forceinline__ float warp_max(float v) {  // NaN counts for nothing
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ void fma2(float &x0, float &x1, float s, float v0, float v1) {  // x += s * v
  asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %2};\n mov.b64 b, {%3, %4};\n mov.b64 c, {%0, %1};\n"
      " fma.rn.f32x2 c, a, b, c;\n mov.b64 {%0, %1}, c;\n}\n"
      : "+f"(x0), "+f"(x1) : "f"(s), "f"(v0), "f"(v1));
}
__device__ __forceinline__ void mul2(float &x0, float &x1, float s, float v0, float v1) {  // x = s * v
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%2, %2};\n mov.b64 b, {%3, %4};\n mul.rn.f32x2 b, a, b;\n"
      " mov.b64 {%0, %1}, b;\n}\n"
      : "=f"(x0), "=f"(x1) : "f"(s), "f"(v0), "f"(v1));
}
__device__ __forceinline__ void fma2(float &x0, float &x1, float s0, float s1, float a0, float a1) {  // x = x * s + a
  asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %3};\n mov.b64 c, {%4, %5};\n"
      " fma.rn.f32x2 c, a, b, c;\n mov.b64 {%0, %1}, c;\n}\n"
      : "+f"(x0), "+f"(x1) : "f"(s0), "f"(s1), "f"(a0), "f"(a1));
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&b);
}
// Sums of N values over a warp's lanes: lane h (and h + N, ...) gets the h-th.  Each step
// sends the half of the values that the other lane will keep.
template <int N>
__device__ __forceinline__ float sum_rows(const float (&v)[N], uint32_t lane) {
  float x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = v[i];
#pragma unroll
  for (int d = N / 2; d; d >>= 1)
#pragma unroll
    for (int i = 0; i < d; ++i) {
      const bool up = lane & d;
      const float keep = up ? x[i + d] : x[i], send = up ? x[i] : x[i + d];
      x[i] = keep + __shfl_xor_sync(0xffffffffu, send, d);
    }
  float r = x[0];
#pragma unroll
  for (int d = N; d < 32; d <<= 1) r += __shfl_xor_sync(0xffffffffu, r, d);
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Shared-memory operand descriptor, 128-byte swizzle (the swizzle XORs bits 4-6 of an
// address with bits 7-9, so every operand region starts on 1,024 bytes).  K-major: rows of
// 64 elements, 8 rows in 1,024 bytes (stride); MN-major: 64 elements of M or N in 128
// bytes, 8 of K in 1,024 bytes (stride), the next 64 of M `lead` bytes on.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(lead >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// e4m3 codes (two in the low half of `two`) to f16 and to bf16, exactly.
__device__ __forceinline__ uint32_t codes_to_f16(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return h;
}
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t two) {
  const uint32_t h = codes_to_f16(two);
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
  return __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);  // (their low halves are 0)
}

}  // namespace ula_tc
