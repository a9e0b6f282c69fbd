// tc_ptx.cuh -- the PTX instructions, bounded waits, operand layouts and
// two-term operand splits that the tensor-core kernels of this library share.
#pragma once
#include <cuda.h>

#include <type_traits>

#include "common.cuh"

namespace gtr {
namespace tc {

constexpr unsigned long long kWaitNs = 500ull * 1000 * 1000;   // bounded waits: 0.5 s

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ uint32_t saddr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ unsigned long long globaltimer() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ void mbar_init(uint64_t* b, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_fence_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
// One bounded probe of a phase; the thread may sleep in hardware for up to
// 20 us while the phase is incomplete (fewer polling instructions).
__device__ __forceinline__ uint32_t mbar_try(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(saddr(b)), "r"(parity), "r"(20000u)
      : "memory");
  return ok;
}
// Wait for the phase with the given parity to complete; false after kWaitNs.
__device__ __forceinline__ bool mbar_wait(uint64_t* b, uint32_t parity) {
  if (mbar_try(b, parity)) return true;
  const unsigned long long t0 = globaltimer();
  while (!mbar_try(b, parity))
    if (globaltimer() - t0 > kWaitNs) return false;
  return true;
}
// One plain arrival.
__device__ __forceinline__ void mbar_arrive_one(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(b)) : "memory");
}
// One arrival that also expects `bytes` of asynchronous copies on the barrier.
__device__ __forceinline__ void mbar_arrive_tx(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(b)), "r"(bytes)
               : "memory");
}
// Tensor-map box loads (global -> shared), completing on an mbarrier.  The
// innermost coordinate is always 0 here (16-byte aligned); the others may be
// negative or past the end, which reads zeros.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
      "%4, %5}], [%6];" ::"r"(saddr(dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(saddr(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                            int c4, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
      "%4, %5, %6}], [%7];" ::"r"(saddr(dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(saddr(bar))
      : "memory");
}
// Tiled tensor-map stores shared -> global (bulk-group completion).  The
// innermost coordinate must be 16-byte aligned and no coordinate negative.
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, const void* src, int c0, int c1, int c2,
                                             int c3) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
                   map),
               "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(saddr(src))
               : "memory");
}
__device__ __forceinline__ void tma_store_5d(const CUtensorMap* map, const void* src, int c0, int c1, int c2,
                                             int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4, %5}], [%6];" ::"l"(map),
      "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(saddr(src))
      : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// wait until at most N committed bulk stores still read shared memory / are in flight
template <int N> __device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
template <int N> __device__ __forceinline__ void bulk_wait() {
  asm volatile("cp.async.bulk.wait_group %0;" ::"n"(N) : "memory");
}
// 16-byte asynchronous global -> shared copy (L2 only), grouped by commit.
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(saddr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// wait until at most N of this thread's committed groups are still in flight
template <int N> __device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void tc_before_sync() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after_sync() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(dst)),
               "r"(cols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols)
               : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(saddr(bar))
      : "memory");
}
// 16 lanes x 32 bit in two halves: thread t of warp w reads lane 32(w%4) + t%16
// of the address's quadrant, columns [c, c+16) for t < 16 and [c+16, c+32) for
// t >= 16 (c = the address's column).
__device__ __forceinline__ void tmem_ld16x2(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16], 16;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// Wait for this thread's tcgen05.ld, tied to the 16 registers of the load so
// that no use of them can be scheduled before it (the compiler does not know
// the load is asynchronous).
__device__ __forceinline__ void tmem_ld_wait(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]),
                 "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]),
                 "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}
// 16 lanes x 32 bit in two halves, eight columns each (the store counterpart
// of tmem_ld16x2 at half the width): thread t of warp w writes lane
// 32(w%4) + t%16, columns [c, c+8) for t < 16 and [c+8, c+16) for t >= 16.
__device__ __forceinline__ void tmem_st8x2(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x32bx2.x8.b32 [%0], 8, {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// barrier over `count` threads (whole warps) on hardware barrier `id` (1..15)
__device__ __forceinline__ void named_barrier(int id, int count) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}
// The same barrier, also OR-ing a predicate across its threads.
__device__ __forceinline__ bool named_barrier_or(int id, int count, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(count), "r"((uint32_t)pred)
      : "memory");
  return r != 0;
}
// 2^x by the hardware approximation (ex2.approx, flush-to-zero)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Power-of-two operand scales: 2^e puts the magnitude m into [2^14, 2^15),
// inside fp16's range; exact, and undone on the fp32 accumulator.
__device__ __forceinline__ int scale_exp(float m) {
  if (!(m > 0.f) || !(m <= 3.0e38f)) return 0;
  const int ex = ((__float_as_int(m) >> 23) & 0xFF) - 127;
  return max(-60, min(60, 14 - ex));
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((127 + e) << 23); }
// Two fp32 lanes per instruction (add / mul / fma .f32x2, sm_100): a pair of
// floats in one 64-bit register, the first in the low half.
__device__ __forceinline__ uint64_t f2pack(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 f2unpack(uint64_t r) {
  float a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
  return make_float2(a, b);
}
__device__ __forceinline__ uint64_t ffma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// Two-term fp16 value pairs: x = hi + lo, hi = fp16(x), lo = fp16(x - hi),
// two consecutive elements per 32-bit word.
__device__ __forceinline__ void split2h(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
  memcpy(&hi, &h, 4);
  memcpy(&lo, &l, 4);
}
// Untiled bulk copy global -> shared (16-byte aligned, size a multiple of 16),
// completing on `bar` (which must expect the bytes).
__device__ __forceinline__ void bulk_g2s(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          saddr(dst)),
      "l"(src), "r"(bytes), "r"(saddr(bar))
      : "memory");
}

// ------------------------------------------------------- operand layouts
// 16-bit operand tiles of 64 rows x 64 elements (128 bytes per row), layout
// SWIZZLE_128B: atoms of 8 rows x 128 bytes, the 16-byte unit index XOR-ed
// with the row's position in its atom.  The same physical layout serves a
// K-major operand (rows = M or N, columns = K) and an MN-major one (rows = K,
// columns = M or N); only the descriptor differs.
__device__ __forceinline__ uint32_t sw_unit(int r, int u) {
  return (uint32_t)((r >> 3) * 1024 + (r & 7) * 128 + ((u ^ (r & 7)) << 4));
}
__device__ __forceinline__ uint32_t sw16(int r, int c) { return sw_unit(r, c >> 3) + (c & 7) * 2; }
// tcgen05 shared-memory matrix descriptor (version 1): start address, leading
// and stride byte offsets, layout type 2 = SWIZZLE_128B.
__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}
// K-major tile: a K step of 16 elements is 32 bytes into every row.
__device__ __forceinline__ uint64_t desc_k(const void* tile) { return sdesc(saddr(tile), 16, 1024); }
// MN-major tile: a K step of 16 rows is two 8-row atoms, 2048 bytes.
__device__ __forceinline__ uint64_t desc_mn(const void* tile) { return sdesc(saddr(tile), 8192, 1024); }
constexpr uint32_t kStepK = 32 >> 4, kStepMN = 2048 >> 4;   // descriptor address units per K step
// Instruction descriptor: kind::f16 with bf16 A and B, fp32 accumulate, M = 64,
// N = n (64 unless given).
__host__ __device__ constexpr uint32_t idesc_bf16(int a_mn, int b_mn, int n = 64) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(64 >> 4) << 24);
}
// The same with fp16 A and B.
__host__ __device__ constexpr uint32_t idesc_f16(int a_mn, int b_mn, int n = 64) {
  return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(64 >> 4) << 24);
}
// One tcgen05.mma kind::f16 instruction; the instruction descriptor selects
// fp16 or bf16 operands.
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// One tcgen05.mma kind::f16 with A in tensor memory (M = 64: row r in lane
// 32 (r / 16) + r % 16, two 16-bit elements per 32-bit column, the even one
// in the low half; a K = 16 step is 8 columns).
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                           uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// d += (ah + al)(bh + bl) ~ ah bh + ah bl + al bh over K = 64, A in tensor memory
template <uint32_t SB>
__device__ __forceinline__ void mma_terms_ts(uint32_t d, uint32_t ah, uint32_t al, uint64_t bh, uint64_t bl,
                                             bool b_two, uint32_t id) {
#pragma unroll
  for (uint32_t s = 0; s < 4; ++s) mma_f16_ts(d, ah + 8 * s, bh + s * SB, id, 1u);
  if (b_two) {
#pragma unroll
    for (uint32_t s = 0; s < 4; ++s) mma_f16_ts(d, ah + 8 * s, bl + s * SB, id, 1u);
  }
#pragma unroll
  for (uint32_t s = 0; s < 4; ++s) mma_f16_ts(d, al + 8 * s, bh + s * SB, id, 1u);
}
// d (+)= A B over K = 64: four K = 16 instructions.
template <uint32_t SA, uint32_t SB>
__device__ __forceinline__ void mma_k64(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool acc) {
#pragma unroll
  for (uint32_t s = 0; s < 4; ++s) mma_f16(d, a + s * SA, b + s * SB, id, (acc || s) ? 1u : 0u);
}
// (ah + al)(bh + bl) ~ ah bh + ah bl + al bh, or ah b + al b for a one-term B.
template <uint32_t SA, uint32_t SB>
__device__ __forceinline__ void mma_terms(uint32_t d, uint64_t ah, uint64_t al, uint64_t bh,
                                          uint64_t bl, bool b_two, uint32_t id, bool acc) {
  mma_k64<SA, SB>(d, ah, bh, id, acc);
  if (b_two) mma_k64<SA, SB>(d, ah, bl, id, true);
  mma_k64<SA, SB>(d, al, bh, id, true);
}
// The same with the optional second term on A: a bh + a bl for a one-term A.
template <uint32_t SA, uint32_t SB>
__device__ __forceinline__ void mma_terms_a(uint32_t d, uint64_t ah, uint64_t al, uint64_t bh,
                                            uint64_t bl, bool a_two, uint32_t id, bool acc) {
  mma_k64<SA, SB>(d, ah, bh, id, acc);
  mma_k64<SA, SB>(d, ah, bl, id, true);
  if (a_two) mma_k64<SA, SB>(d, al, bh, id, true);
}

// --------------------------------------------------- two-term bf16 operands
__device__ __forceinline__ uint32_t bits2(__nv_bfloat162 h) {
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  const float2 f = __bfloat1622float2(h);
  hi = bits2(h);
  lo = bits2(__floats2bfloat162_rn(a - f.x, b - f.y));   // a - hi is exact in fp32
}
// four consecutive elements (8 bytes) at byte offset `off` of the (hi, lo) tiles
__device__ __forceinline__ void put4(uint8_t* H, uint8_t* L, uint32_t off, float a, float b, float c,
                                     float d) {
  uint32_t h0, l0, h1, l1;
  split2(a, b, h0, l0);
  split2(c, d, h1, l1);
  *reinterpret_cast<uint2*>(H + off) = make_uint2(h0, h1);
  *reinterpret_cast<uint2*>(L + off) = make_uint2(l0, l1);
}

// eight consecutive elements (16 bytes, one swizzle unit) at byte offset `off`
__device__ __forceinline__ void put8(uint8_t* H, uint8_t* L, uint32_t off, const float* x) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) split2(x[2 * i], x[2 * i + 1], h[i], l[i]);
  *reinterpret_cast<uint4*>(H + off) = make_uint4(h[0], h[1], h[2], h[3]);
  *reinterpret_cast<uint4*>(L + off) = make_uint4(l[0], l[1], l[2], l[3]);
}

// two consecutive elements (4 bytes) at byte offset `off` of the (hi, lo) tiles
// the same in fp16 terms
__device__ __forceinline__ void put2h(uint8_t* H, uint8_t* L, uint32_t off, float a, float b) {
  uint32_t h, l;
  split2h(a, b, h, l);
  *reinterpret_cast<uint32_t*>(H + off) = h;
  *reinterpret_cast<uint32_t*>(L + off) = l;
}
__device__ __forceinline__ void put2x(uint8_t* H, uint8_t* L, uint32_t off, float a, float b) {
  uint32_t h, l;
  split2(a, b, h, l);
  *reinterpret_cast<uint32_t*>(H + off) = h;
  *reinterpret_cast<uint32_t*>(L + off) = l;
}

template <typename T> struct Vec4;
template <> struct Vec4<__half> {
  static __device__ __forceinline__ float4 from_bits(uint2 u) {
    __half2 a, b;
    memcpy(&a, &u.x, 4);
    memcpy(&b, &u.y, 4);
    const float2 fa = __half22float2(a), fb = __half22float2(b);
    return make_float4(fa.x, fa.y, fb.x, fb.y);
  }
  static __device__ __forceinline__ float4 load(const void* p) {
    return from_bits(*reinterpret_cast<const uint2*>(p));
  }
};
template <> struct Vec4<__nv_bfloat16> {
  static __device__ __forceinline__ float4 from_bits(uint2 u) {
    __nv_bfloat162 a, b;
    memcpy(&a, &u.x, 4);
    memcpy(&b, &u.y, 4);
    const float2 fa = __bfloat1622float2(a), fb = __bfloat1622float2(b);
    return make_float4(fa.x, fa.y, fb.x, fb.y);
  }
  static __device__ __forceinline__ float4 load(const void* p) {
    return from_bits(*reinterpret_cast<const uint2*>(p));
  }
};
// two consecutive 16-bit elements as floats
__device__ __forceinline__ float2 ld2(const __half* p) { return __half22float2(*reinterpret_cast<const __half2*>(p)); }
__device__ __forceinline__ float2 ld2(const __nv_bfloat16* p) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
}

template <typename T> __device__ __forceinline__ uint2 pack4(float a, float b, float c, float d);
template <> __device__ __forceinline__ uint2 pack4<__half>(float a, float b, float c, float d) {
  const __half2 x = __floats2half2_rn(a, b), y = __floats2half2_rn(c, d);
  uint2 u;
  memcpy(&u.x, &x, 4);
  memcpy(&u.y, &y, 4);
  return u;
}
template <> __device__ __forceinline__ uint2 pack4<__nv_bfloat16>(float a, float b, float c, float d) {
  return make_uint2(bits2(__floats2bfloat162_rn(a, b)), bits2(__floats2bfloat162_rn(c, d)));
}

}  // namespace tc
}  // namespace gtr
