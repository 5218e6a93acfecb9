// Inline PTX of the tensor-core attention kernels: mbarriers with bounded
// waits, TMA tile loads, and the tcgen05 matrix unit with its tensor memory.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace fm {
namespace tc {

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// ---- mbarriers --------------------------------------------------------------
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
// the memory of a barrier that nothing uses any more, for another
__device__ __forceinline__ void bar_free(uint32_t bar) {
  asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
// Where a wait that gave up is noted: in a word on the device, which other waits
// look at while they poll, and in one in host memory, which the next call looks at.
struct ErrorWords {
  unsigned *device, *host;
};
// A wait that ends: after two seconds or 2^26 polls it gives up, records the
// error and returns false, and so does every wait that finds the error (its
// own block's flag, or the device's word) while it polls. A role that got
// false runs to its end without touching tensor memory or issuing copies.
__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity, volatile int* dead, const ErrorWords& err) {
  const unsigned long long begin = now_ns();
#pragma unroll 1
  for (int i = 0; i < (1 << 20); ++i) {
#pragma unroll 1
    for (int k = 0; k < 64; ++k)
      if (bar_try(bar, parity)) return true;
    if (*dead) return false;
    if (*(volatile unsigned*)err.device != 0 || now_ns() - begin > 2000000000ull) break;
  }
  *dead = 1;
  atomicExch(err.device, 5u /* FM_ERR_KERNEL_TIMEOUT */);
  *(volatile unsigned*)err.host = 5u;
  __threadfence_system();
  return false;
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* dead, const ErrorWords& err) {
#pragma unroll 1
  for (int k = 0; k < 32; ++k)
    if (bar_try(bar, parity)) return true;
  return bar_wait_slow(bar, parity, dead, err);
}

// ---- TMA --------------------------------------------------------------------
__device__ __forceinline__ void tma_prefetch(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}
// box of 64 elements x rows x 1 x 1 at {x, token, head, batch}
__device__ __forceinline__ void tma_load(uint32_t to, const CUtensorMap* m, uint32_t bar, int x, int t, int h, int b) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];" ::"r"(to),
      "l"(m), "r"(bar), "r"(x), "r"(t), "r"(h), "r"(b)
      : "memory");
}
// orders this thread's shared-memory writes before later reads by the
// asynchronous units (TMA, tcgen05)
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void fence_bar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// ---- tensor memory ----------------------------------------------------------
// once in a block's life: after giving the permit up it may allocate no more
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define FM_R8(b, o) "=r"(b[o]), "=r"(b[o + 1]), "=r"(b[o + 2]), "=r"(b[o + 3]), "=r"(b[o + 4]), "=r"(b[o + 5]), "=r"(b[o + 6]), "=r"(b[o + 7])
#define FM_I8(b, o) "r"(b[o]), "r"(b[o + 1]), "r"(b[o + 2]), "r"(b[o + 3]), "r"(b[o + 4]), "r"(b[o + 5]), "r"(b[o + 6]), "r"(b[o + 7])
#define FM_P8(b, o) "+r"(b[o]), "+r"(b[o + 1]), "+r"(b[o + 2]), "+r"(b[o + 3]), "+r"(b[o + 4]), "+r"(b[o + 5]), "+r"(b[o + 6]), "+r"(b[o + 7])

// 32 columns of this warp's 32 lanes: thread t gets lane t's row
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : FM_R8(r, 0), FM_R8(r, 8), FM_R8(r, 16), FM_R8(r, 24)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : FM_R8(r, 0), FM_R8(r, 8)
      : "r"(addr)
      : "memory");
}
// ties loaded registers to the wait before it: what uses them stays behind
__device__ __forceinline__ void tie32(uint32_t* r) {
  asm volatile("" : FM_P8(r, 0), FM_P8(r, 8), FM_P8(r, 16), FM_P8(r, 24)::"memory");
}
__device__ __forceinline__ void tie16(uint32_t* r) { asm volatile("" : FM_P8(r, 0), FM_P8(r, 8)::"memory"); }
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::FM_I8(r, 0),
      FM_I8(r, 8), FM_I8(r, 16), FM_I8(r, 24), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15};" ::FM_I8(r, 0),
      FM_I8(r, 8), "r"(addr)
      : "memory");
}

// ---- matrix products --------------------------------------------------------
// Shared-memory operands are tiles of 128-byte rows with the 128-byte swizzle
// that TMA writes: 8 rows make a 1024-byte group, groups follow one another.
// K-major (the summed index runs along the row): a step of 16 elements is 32
// bytes further. MN-major (the summed index runs over rows): a step of 16 is
// two groups, 2048 bytes, further, and `across` is the distance between
// tiles of 64 columns.
constexpr uint64_t kDescCommon = (uint64_t)1 << 46 | (uint64_t)2 << 61;
__device__ __forceinline__ uint64_t desc_k(uint32_t addr) {
  return kDescCommon | (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32;
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t across) {
  return kDescCommon | (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)(across >> 4) << 16 |
         (uint64_t)(1024 >> 4) << 32;
}
// f32 accumulators; A and B both bf16 or both f16; B K-major or MN-major
__device__ __forceinline__ uint32_t instr_desc(int m, int n, bool bf16, bool b_mn) {
  return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (b_mn ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 |
         (uint32_t)(m >> 4) << 24;
}
// Products are issued by a whole converged warp, of which one lane (`lead`)
// executes them: addresses and descriptors then stay in uniform registers.
// Issued from one lane's own branch they cost about a hundred cycles each.
__device__ __forceinline__ uint32_t elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"(lead)
      : "memory");
}
// arrives on bar once every product issued so far by this thread is done
__device__ __forceinline__ void mma_commit(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.u32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(lead)
      : "memory");
}

// ---- registers of a group of four warps -------------------------------------
template <int N>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ---- arithmetic -------------------------------------------------------------
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// tanh(x) = 1 - 2 / (e^2x + 1) from x2 = 2 log2(e) x. Saturates cleanly at both
// ends, but its error is absolute (about 2^-22): times a large cap it would
// swamp the scores far below the cap. So it is for |x| > kTanhSmall only, where
// tanh(x) is large enough for it.
__device__ __forceinline__ float tanh_from(float x2) { return fmaf(-2.f, rcp(ex2(x2) + 1.f), 1.f); }
// Below that, tanh(x) / x is a polynomial of degree 3 in x^2, fitted for the
// least relative error there (1e-7).
constexpr float kTanhSmall = 0.4f;
__device__ __forceinline__ float tanh_over_x(int i) {
  constexpr float a[4] = {0.999999902f, -0.333313625f, 0.132709768f, -0.0475536036f};
  return a[i];
}

// pairs of 32-bit floats in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// what packing took from each of the two
template <bool BF16>
__device__ __forceinline__ uint32_t rest2(float lo, float hi, uint32_t packed) {
  float a, z;
  if (BF16) {
    a = __uint_as_float(packed << 16);
    z = __uint_as_float(packed & 0xffff0000u);
  } else {
    const __half2 h = *reinterpret_cast<const __half2*>(&packed);
    a = __low2float(h);
    z = __high2float(h);
  }
  return pack2<BF16>(lo - a, hi - z);
}

}  // namespace tc
}  // namespace fm
