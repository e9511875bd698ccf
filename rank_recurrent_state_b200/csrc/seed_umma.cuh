// seed_umma.cuh -- tcgen05 (5th-generation tensor core) primitives as inline PTX for
// sm_100a, and the two-term fp16 form in which float32 operands reach it.
//
// A float32 product on the tensor cores: each operand is scaled by a power of two (per
// row, so that the row's largest value lies in [1, 2)), split as x = hi + lo in fp16,
// and multiplied as lo hi + hi lo + hi hi with float32 accumulation.  hi is off by at
// most 2^-11 of the row's scale, lo by 2^-25 (fp16's subnormal step is 2^-24), and the
// dropped lo lo is below 2^-22: the products are accurate to about 2^-22 of the rows'
// scales, as float32 FMA chains are, at a third of the fp16 rate.  Scaling and its
// undoing are exact.
#pragma once

#include "seed_tma.cuh"

namespace seed {

// ------------------------------------------------------------------ tensor memory
// 32-bit address: lane in bits 16..31, column in bits 0..15.
SEED_DEV void tmem_alloc(uint32_t* smem_slot, uint32_t cols) {      // one warp, all lanes
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(smem_slot)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
SEED_DEV void tmem_free(uint32_t addr, uint32_t cols) {             // the same warp
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
SEED_DEV void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
SEED_DEV void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
SEED_DEV void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
SEED_DEV void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 consecutive columns of the warp's 32 lanes (lane base 32 (warp % 4) in addr).
SEED_DEV void tmem_ld16(uint32_t addr, float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
      : "r"(addr)
      : "memory");
}
SEED_DEV void tmem_st8(uint32_t addr, const uint32_t* u) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(u[0]),
               "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
               : "memory");
}

// ------------------------------------------------------------------ descriptors
// Shared-memory operand tiles: 128-byte rows in the 128-byte swizzle (the 16-byte chunk
// index is xor-ed with the row index mod 8), 1024-byte aligned.
//   K-major:  rows run along N, a row holds 64 consecutive K; 8-row groups 1024 B apart
//   MN-major: rows run along K, a row holds 64 consecutive N; the next 64 N `panel` bytes on
SEED_DEV uint64_t umma_desc(uint32_t saddr, uint32_t lbo_bytes) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3ffffu) >> 4);
  d |= (uint64_t)(lbo_bytes >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;      // stride between 8-row groups
  d |= (uint64_t)1 << 46;                 // descriptor version of sm_100
  d |= (uint64_t)2 << 61;                 // 128-byte swizzle
  return d;
}
// fp16 x fp16 -> float32; bit 16: B is MN-major.
constexpr uint32_t umma_idesc(int M, int N, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// D[tmem] (+)= A[tmem] B[smem], one k-step of 16; issued by one thread.
SEED_DEV void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
// Same with A in shared memory (K-major tile).
SEED_DEV void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
// Arrives once on the barrier when every product issued so far by this thread is done.
SEED_DEV void umma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}

SEED_DEV void named_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

// ------------------------------------------------------------------ two-term fp16
// 2^-e for the power of two 2^e <= m < 2^(e+1) (1 for a zero or non-finite m, so that
// those go through unchanged), kept where both it and its inverse are normal numbers.
SEED_DEV float pow2_scale(float m) {
  const int e = (int)((__float_as_uint(m) >> 23) & 0xffu);
  if (e == 0 || e == 255) return 1.f;
  const int s = 254 - e;                            // exponent field of 2^-(e - 127)
  return __uint_as_float((uint32_t)(s < 1 ? 1 : s) << 23);
}
SEED_DEV float pow2_inverse(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

// Two float32 operations in one instruction.
SEED_DEV uint64_t pack2(float2 a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
SEED_DEV float2 unpack2(uint64_t a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
SEED_DEV float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack2(a)), "l"(pack2(b)));
  return unpack2(r);
}
SEED_DEV float2 mul2(float2 a, float b) { return mul2(a, make_float2(b, b)); }
SEED_DEV float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pack2(a)), "l"(pack2(b)), "l"(pack2(c)));
  return unpack2(r);
}

SEED_DEV void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 d = fma2(__half22float2(h), make_float2(-1.f, -1.f), make_float2(x, y));      // exact
  const __half2 l = __floats2half2_rn(d.x, d.y);
  memcpy(&hi, &h, 4);
  memcpy(&lo, &l, 4);
}
SEED_DEV void split2_scaled(float x, float y, float s, uint32_t& hi, uint32_t& lo) {
  const float2 a = mul2(make_float2(x, y), s);
  split2(a.x, a.y, hi, lo);
}

}  // namespace seed
