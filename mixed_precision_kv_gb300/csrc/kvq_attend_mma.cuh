// Device parts shared by the two tensor-core kernels of kv_attend: barriers
// with bounded waits, tcgen05 wrappers, and the dequantization of page blocks
// to binary16 pairs.
//
// Order of elements.  Both kernels contract over channels (Q K^T) and over
// tokens (P V), and the order inside a contraction is free as long as both
// operands share it.  The order taken is the one the code words unpack to: the
// 8 channels of a K code word (and the 8 slots of a V code word) come out as
// the pairs (n, n + 4), n = 0..3, so element n of a run of 8 sits at
//     order8(n) = 2 * (n & 3) + (n >> 2).
// A 32-bit word of two binary16 values never has to be repacked.
//
// Unpacking.  A code field at bits p.. of both halves or-ed with 0x6400 is
// binary16 1024 + code * 2^p, exactly; one fused multiply-add takes it to the
// code (exact) and a second to code * scale + zero, rounded once to binary16:
// relative 2^-11 of the value, against the 2^-8 of the bf16 result.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq_attend.h"

namespace kvq {
namespace {

constexpr uint32_t kAttSpin = 1u << 22;   // bound of every wait, in polls

__device__ __forceinline__ uint32_t sm32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// ---- barriers --------------------------------------------------------------
__device__ __forceinline__ void mb_init(uint64_t* b, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(sm32(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void mb_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(sm32(b)) : "memory");
}
__device__ __forceinline__ bool mb_try(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok) : "r"(sm32(b)), "r"(parity) : "memory");
  return ok != 0;
}
// Wait for the phase of `parity`; false once `limit` polls are used up or
// another role gave up (then every role leaves its loop).
__device__ __forceinline__ bool mb_wait(uint64_t* b, uint32_t parity, volatile uint32_t* gave_up,
                                        uint32_t limit = kAttSpin) {
  for (uint32_t it = 0; it < limit; ++it) {
    if (mb_try(b, parity)) return true;
    if (*gave_up) return false;
  }
  *gave_up = 1u;
  return false;
}
// The same without suspending the thread: for the one wait on the critical path of a
// single thread (2048 tokens over 32K: 1.76 ms, 1.78 without).  Whole warps that spin
// take issue slots from the others (1.82 ms).
__device__ __forceinline__ bool mb_spin(uint64_t* b, uint32_t parity, volatile uint32_t* gave_up) {
  for (uint32_t it = 0; it < (1u << 26); ++it) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok) : "r"(sm32(b)), "r"(parity) : "memory");
    if (ok) return true;
    if ((it & 63u) == 63u && *gave_up) return false;
  }
  *gave_up = 1u;
  return false;
}
__device__ __forceinline__ void bulk_to_smem(void* dst, const void* src, uint32_t bytes, uint64_t* b) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the slot was read generically
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(sm32(b)), "r"(bytes) : "memory");
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(sm32(dst)), "l"(src), "r"(bytes), "r"(sm32(b)) : "memory");
}

// ---- tcgen05 ---------------------------------------------------------------
__device__ __forceinline__ void tm_alloc(uint32_t* slot, uint32_t cols) {   // one warp
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sm32(slot)), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tm_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void tm_commit(uint64_t* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(sm32(b)) : "memory");
}
__device__ __forceinline__ void tm_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// D[tmem] (+)= A B^T, binary16 operands, fp32 sums; A from shared memory or from TMEM
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
               " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
               ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
               " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
               ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
// fp32 accumulator, binary16 operands, both K-major; M rows of A, N rows of B
__host__ __device__ constexpr uint32_t mma_idesc(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// K-major operand in 128-byte swizzled rows (8-row atoms of 1024 bytes)
__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t(1) << 16) | (uint64_t(64) << 32) | (uint64_t(1) << 46) |
         (uint64_t(2) << 61);
}
// Byte offset of 16-byte chunk c (0..15) of row r in an operand tile of 128
// elements per row: two blocks of `rows` 128-byte rows, chunks swizzled.
__device__ __forceinline__ uint32_t tile_off(int rows, int r, int c) {
  return (uint32_t)((c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
template <int N>
__device__ __forceinline__ void tm_ld(uint32_t (&r)[N], uint32_t addr);   // 32 lanes x N columns, lane = thread
template <>
__device__ __forceinline__ void tm_ld<8>(uint32_t (&r)[8], uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "r"(addr));
}
template <>
__device__ __forceinline__ void tm_ld<16>(uint32_t (&r)[16], uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                 "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(addr));
}
template <>
__device__ __forceinline__ void tm_ld<32>(uint32_t (&r)[32], uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
               "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                 "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                 "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                 "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
               : "r"(addr));
}
// 32 columns into r[kAt ..] of a longer array
template <int kAt, int N>
__device__ __forceinline__ void tm_ld32_at(uint32_t (&r)[N], uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
               : "=r"(r[kAt+0]), "=r"(r[kAt+1]), "=r"(r[kAt+2]), "=r"(r[kAt+3]), "=r"(r[kAt+4]), "=r"(r[kAt+5]), "=r"(r[kAt+6]), "=r"(r[kAt+7]), "=r"(r[kAt+8]), "=r"(r[kAt+9]), "=r"(r[kAt+10]), "=r"(r[kAt+11]), "=r"(r[kAt+12]), "=r"(r[kAt+13]), "=r"(r[kAt+14]), "=r"(r[kAt+15]), "=r"(r[kAt+16]), "=r"(r[kAt+17]), "=r"(r[kAt+18]), "=r"(r[kAt+19]), "=r"(r[kAt+20]), "=r"(r[kAt+21]), "=r"(r[kAt+22]), "=r"(r[kAt+23]), "=r"(r[kAt+24]), "=r"(r[kAt+25]), "=r"(r[kAt+26]), "=r"(r[kAt+27]), "=r"(r[kAt+28]), "=r"(r[kAt+29]), "=r"(r[kAt+30]), "=r"(r[kAt+31])
               : "r"(addr));
}
template <int N>
__device__ __forceinline__ void tm_st(uint32_t addr, const uint32_t (&r)[N]);
template <>
__device__ __forceinline__ void tm_st<8>(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}
template <>
__device__ __forceinline__ void tm_st<16>(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
               ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                 "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}

// ---- arithmetic ------------------------------------------------------------
__device__ __forceinline__ float ex2f(float x) {   // 2^x; results below 2^-126 are 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t hfma2u(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t hadd2u(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hmul2u(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// (a0, a1) * (b0, b1) + (c0, c1), each rounded once
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1, float c0, float c1) {
  asm("{.reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 a, a, b, c;\n mov.b64 {%0, %1}, a;}"
      : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void add2f(float& a0, float& a1, float b0, float b1) {
  asm("{.reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n add.rn.f32x2 x, x, y;\n"
      " mov.b64 {%0, %1}, x;}"
      : "+f"(a0), "+f"(a1) : "f"(b0), "f"(b1));
}
// (x & mask) | 0x64006400
template <uint32_t kMask>
__device__ __forceinline__ uint32_t field(uint32_t x) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(x), "n"(kMask), "n"(0x64006400u));
  return d;
}
// a pair of codes at bits 0, 2, 4 or 6 of both halves as binary16 (exact)
__device__ __forceinline__ uint32_t codes0(uint32_t f) { return hadd2u(f, 0xE400E400u); }                 // - 1024
__device__ __forceinline__ uint32_t codes2(uint32_t f) { return hfma2u(f, 0x34003400u, 0xDC00DC00u); }    // / 4 - 256
__device__ __forceinline__ uint32_t codes4(uint32_t f) { return hfma2u(f, 0x2C002C00u, 0xD400D400u); }    // / 16 - 64
__device__ __forceinline__ uint32_t codes6(uint32_t f) { return hfma2u(f, 0x24002400u, 0xCC00CC00u); }    // / 64 - 16
// the 8 nibbles of a word: pairs (k, k + 4)
__device__ __forceinline__ void nibbles(uint32_t x, uint32_t (&c)[4]) {
  const uint32_t y = x >> 8;
  c[0] = codes0(field<0x000F000Fu>(x));
  c[1] = codes4(field<0x00F000F0u>(x));
  c[2] = codes0(field<0x000F000Fu>(y));
  c[3] = codes4(field<0x00F000F0u>(y));
}
// 2-bit fields at bits 0, 2, 4, 6 of both halves
__device__ __forceinline__ void crumbs(uint32_t x, uint32_t (&c)[4]) {
  c[0] = codes0(field<0x00030003u>(x));
  c[1] = codes2(field<0x000C000Cu>(x));
  c[2] = codes4(field<0x00300030u>(x));
  c[3] = codes6(field<0x00C000C0u>(x));
}
// a byte of two E2M1 codes as binary16 values
__device__ __forceinline__ uint32_t e2m1x2(uint32_t x) {
  uint32_t d;
  asm("{.reg .b8 t;\n cvt.u8.u32 t, %1;\n cvt.rn.f16x2.e2m1x2 %0, t;\n}" : "=r"(d) : "r"(x));
  return d;
}
__device__ __forceinline__ int order8(int n) { return 2 * (n & 3) + (n >> 2); }
// bits of 32 slots in the order of the operand tiles
__device__ __forceinline__ uint32_t order_bits(uint32_t m) {
  uint32_t d = 0u;
#pragma unroll
  for (int n = 0; n < 8; ++n) d |= ((m >> n) & 0x01010101u) << (2 * (n & 3) + (n >> 2));
  return d;
}

// ---- K of a page: slot t, channels 32 gr + 8 i .. + 7 (run (gr, i)) ---------
// out[..][k] = channels (k, k + 4) of a run.
// INT2: the scale and zero pairs of run (gr, i) are the same for every slot.
__device__ __forceinline__ void k_scales2(const uint8_t* blk, int gr, int i, uint32_t (&sc)[4], uint32_t (&z)[4]) {
  const uint32_t sel = (i & 1) ? 0x7632u : 0x5410u, sel0 = (i & 1) ? 0x7610u : 0x5432u;   // pair 0 is stored swapped
  const uint4* p = reinterpret_cast<const uint4*>(blk + kI2KMeta + 4 * ((gr * 2 + (i >> 1)) * 8));
  const uint4 a = p[0], b = p[1], c = p[16], d = p[17];   // zeros 256 bytes on
  sc[0] = __byte_perm(a.x, b.x, sel0);
  sc[1] = __byte_perm(a.y, b.y, sel);
  sc[2] = __byte_perm(a.z, b.z, sel);
  sc[3] = __byte_perm(a.w, b.w, sel);
  z[0] = __byte_perm(c.x, d.x, sel0);
  z[1] = __byte_perm(c.y, d.y, sel);
  z[2] = __byte_perm(c.z, d.z, sel);
  z[3] = __byte_perm(c.w, d.w, sel);
}
__device__ __forceinline__ void k_run2(const uint8_t* blk, int t, int gr, int i, const uint32_t (&sc)[4],
                                       const uint32_t (&z)[4], uint32_t (&out)[4]) {
  const uint32_t h = *reinterpret_cast<const uint16_t*>(blk + kI2KCodes + 32 * t + 8 * gr + 2 * i);
  uint32_t c[4];
  crumbs(__byte_perm(h, 0u, 0x4140u), c);
#pragma unroll
  for (int k = 0; k < 4; ++k) out[k] = hfma2u(c[k], sc[k], z[k]);
}
// The other widths: groups 2 half and 2 half + 1 of slot t.
__device__ __forceinline__ void k_slot4(const uint8_t* blk, int t, int i, int half, uint32_t (&out)[2][4]) {
  const uint2 w = *reinterpret_cast<const uint2*>(blk + kI4KCodes + 64 * t + 16 * i + 8 * half);
  const uint2 m = *reinterpret_cast<const uint2*>(blk + kI4KMeta + 16 * t + 8 * half);
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const uint32_t md = x ? m.y : m.x;
    const uint32_t s = __byte_perm(md, 0u, 0x1010u), z = __byte_perm(md, 0u, 0x3232u);
    uint32_t c[4];
    nibbles(x ? w.y : w.x, c);
#pragma unroll
    for (int k = 0; k < 4; ++k) out[x][k] = hfma2u(c[k], s, z);
  }
}
__device__ __forceinline__ void k_slot3(const uint8_t* blk, int t, int i, int half, uint32_t (&out)[2][4]) {
  const uint32_t lo = *reinterpret_cast<const uint32_t*>(blk + kI3KCodes + 48 * t + 8 * i + 4 * half);
  const uint32_t hi = *reinterpret_cast<const uint32_t*>(blk + kI3KCodes + 48 * t + 32 + 4 * i) >> (8 * half);
  const uint2 m = *reinterpret_cast<const uint2*>(blk + kI3KMeta + 16 * t + 8 * half);
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const uint32_t md = x ? m.y : m.x;
    const uint32_t s = __byte_perm(md, 0u, 0x1010u), z = __byte_perm(md, 0u, 0x3232u);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t c = ((lo >> (8 * x + 2 * k)) & 0x00030003u) | (((hi >> (4 * x + k)) & 0x00010001u) << 2);
      out[x][k] = hfma2u(codes0(c | 0x64006400u), s, z);
    }
  }
}
__device__ __forceinline__ void k_slotf(const uint8_t* blk, int t, int i, int half, uint32_t (&out)[2][4]) {
  const uint2 w = *reinterpret_cast<const uint2*>(blk + kF4KCodes + 64 * t + 16 * i + 8 * half);
  const uint32_t m = *reinterpret_cast<const uint32_t*>(blk + kF4KScale + 8 * t + 4 * half);
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const uint32_t s = __byte_perm(m, 0u, x ? 0x3232u : 0x1010u);
#pragma unroll
    for (int k = 0; k < 4; ++k) out[x][k] = hmul2u(e2m1x2((x ? w.y : w.x) >> (8 * k)), s);
  }
}

// ---- V of a page: channels 32 gr + 8 w + r (w = 0..3), slots 8 i .. 8 i + 7 -
// out[w][k] = slots (k, k + 4) of that run.
__device__ __forceinline__ void v_scales(const uint8_t* blk, int meta, int gr, int i, uint32_t (&s)[4], uint32_t (&z)[4]) {
  const uint4 a = *reinterpret_cast<const uint4*>(blk + meta + 64 * gr + 16 * i);
  const uint4 b = *reinterpret_cast<const uint4*>(blk + meta + 256 + 64 * gr + 16 * i);
  s[0] = a.x; s[1] = a.y; s[2] = a.z; s[3] = a.w;
  z[0] = b.x; z[1] = b.y; z[2] = b.z; z[3] = b.w;
}
__device__ __forceinline__ void v_group4(const uint8_t* blk, int gr, int r, int i, uint32_t (&out)[4][4]) {
  const uint4 w = *reinterpret_cast<const uint4*>(blk + kI4VCodes + 16 * (32 * gr + 4 * r + i));
  const uint32_t wd[4] = {w.x, w.y, w.z, w.w};
  uint32_t s[4], z[4];
  v_scales(blk, kI4VMeta, gr, i, s, z);
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    uint32_t c[4];
    nibbles(wd[x], c);
#pragma unroll
    for (int k = 0; k < 4; ++k) out[x][k] = hfma2u(c[k], s[k], z[k]);
  }
}
__device__ __forceinline__ void v_group2(const uint8_t* blk, int gr, int r, int i, uint32_t (&out)[4][4]) {
  const uint2 w = *reinterpret_cast<const uint2*>(blk + kI2VCodes + 16 * (32 * (gr >> 1) + 4 * r + i) + 8 * (gr & 1));
  uint32_t s[4], z[4];
  v_scales(blk, kI2VMeta, gr, i, s, z);
#pragma unroll
  for (int x = 0; x < 4; ++x) {   // channel 16 (x >> 1) + 8 (x & 1) + r of the group
    const uint32_t wd = (x >> 1) ? w.y : w.x;
    uint32_t c[4];
    crumbs((x & 1) ? wd >> 8 : wd, c);
    if (!(x & 1)) c[0] = __byte_perm(c[0], 0u, 0x1032u);   // slots 8 i and 8 i + 4 are stored swapped
#pragma unroll
    for (int k = 0; k < 4; ++k) out[x][k] = hfma2u(c[k], s[k], z[k]);
  }
}
__device__ __forceinline__ void v_group3(const uint8_t* blk, int gr, int r, int i, uint32_t (&out)[4][4]) {
  const int X = 32 * gr + 4 * r + i;
  const uint2 lo = *reinterpret_cast<const uint2*>(blk + kI3VCodes + 8 * X);
  const uint32_t hi = *reinterpret_cast<const uint32_t*>(blk + kI3VHigh + 4 * X);
  uint32_t s[4], z[4];
  v_scales(blk, kI3VMeta, gr, i, s, z);
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const uint32_t l = ((x >> 1) ? lo.y : lo.x) >> (8 * (x & 1));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t c = ((l >> (2 * k)) & 0x00030003u) | (((hi >> (4 * x + k)) & 0x00010001u) << 2);
      out[x][k] = hfma2u(codes0(c | 0x64006400u), s[k], z[k]);
    }
  }
}
__device__ __forceinline__ void v_groupf(const uint8_t* blk, int gr, int r, int i, uint32_t (&out)[4][4]) {
  const uint4 w = *reinterpret_cast<const uint4*>(blk + kF4VCodes + 16 * (32 * gr + 4 * r + i));
  const uint32_t wd[4] = {w.x, w.y, w.z, w.w};
  const uint4 a = *reinterpret_cast<const uint4*>(blk + kF4VScale + 64 * gr + 16 * i);
  const uint32_t s[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int x = 0; x < 4; ++x)
#pragma unroll
    for (int k = 0; k < 4; ++k) out[x][k] = hmul2u(e2m1x2(wd[x] >> (8 * k)), s[k]);
}

// ---- bf16 rows (full-precision lists, new tokens) --------------------------
__device__ __forceinline__ float bf_f(uint32_t x) { return __uint_as_float(x << 16); }
// a bf16 value for a binary16 operand: NaN, Inf and |x| > 65504 are used as 0 and reported
__device__ __forceinline__ float in_range(float f, uint32_t& bad) {
  if (fabsf(f) <= 65504.0f) return f;
  bad = 1u;
  return 0.0f;
}
// 8 bf16 values at p (2-byte aligned; one 16-byte load where the caller knows p to be 16-byte aligned)
__device__ __noinline__ uint4 load8_unaligned(const uint16_t* p) {
  uint32_t x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = (uint32_t)__ldg(p + 2 * k) | ((uint32_t)__ldg(p + 2 * k + 1) << 16);
  return make_uint4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ uint4 load8(const uint16_t* p, bool aligned) {
  return aligned ? __ldg(reinterpret_cast<const uint4*>(p)) : load8_unaligned(p);
}
// Power-of-two scale of a row of q: exponent e so that mx 2^e lies in [2^7, 2^8)
// (0 for a row that is zero or not finite; at most 126, so that 2^-e is a normal
// number: rows below 2^-119 end below 2^7).
__device__ __forceinline__ int q_exponent(float mx) {
  return mx > 0.0f && mx < INFINITY ? min(126, 134 - (int)(__float_as_uint(mx) >> 23)) : 0;
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// The factor of a row of q: 2^e with the scale's sign.  A row with an infinity (mx; a NaN is
// none) becomes NaN throughout: its logits of keys of one sign could all be -inf otherwise,
// and a row without weight is 0.
__device__ __forceinline__ float q_factor(float mx, int e, float scale) {
  return mx < INFINITY ? copysignf(pow2f(e), scale) : __int_as_float(0x7FFFFFFF);
}
// Rows of a unit: row / g and the row's offset in q and out.  g <= 8, so the high
// word of row * ceil(2^32 / g) is the quotient for every row below 2^29.
struct RowMap {
  uint32_t magic;
  int g;
  __device__ __forceinline__ explicit RowMap(int g_) : magic(0xFFFFFFFFu / (uint32_t)g_ + 1u), g(g_) {}
  __device__ __forceinline__ int token(int row) const { return g == 1 ? row : (int)__umulhi((uint32_t)row, magic); }
  __device__ __forceinline__ size_t at(const AttArgs& A, const AttUnit& u, int row) const {
    const int t = token(row);
    return ((size_t)(u.tok0 + t) * A.hq + (size_t)(u.kvh * g + row - t * g)) * kHeadDim;
  }
};
// 8 values in order8, scaled by 2^e exactly (mul), as binary16
__device__ __forceinline__ void order8_f16(const uint4& x, float mul, uint32_t (&out)[4], uint32_t& bad) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float f[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = in_range(bf_f(w[k] & 0xFFFFu) * mul, bad);
    f[2 * k + 1] = in_range(__uint_as_float(w[k] & 0xFFFF0000u) * mul, bad);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) out[k] = f16x2(f[k], f[k + 4]);
}

}  // namespace
}  // namespace kvq
