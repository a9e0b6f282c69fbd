// hla_tc.cuh -- the tensor-core (tcgen05) kernels of the head-decay linear
// attention for prompts: 16-bit q, k, v, dk and dv of 64 or 128.
//
// Blocks of C = 128 tokens.  With l_t the log-decay of token t of a block, G_i
// the inclusive sum of l up to token i, S the state before the block,
//
//   o_i = e^{G_i} q_i S + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j
//   S  <- e^{G_C} S + sum_j k_j^T (e^{G_C - G_j} v_j)
//
// every factor at most one, so nothing overflows whatever the decays.  No weight
// is a difference of sums from the block's start, which strong decays before both
// tokens would leave few bits of (a reset every fourth token: 2^-11): G_C - G_j is
// a suffix sum of its own; e^{G_i - G_j} is e^{G_i - G_b} e^{G_b - G_j} through the
// end b of j's 32 tokens where i is past it, either sum taken over just the tokens
// in between (one exponential per row and 16 columns); and in the 32 x 32 squares
// on the diagonal it is the product of the decays in between, column by column
// from right to left.
//
// Four matrix products per block, accumulated in fp32 in tensor memory, with
// q, k and v as they are and every computed operand in 16-bit terms (x = hi +
// lo [+ lo2], each the rounding of what is left):
//   scores  = q k^T             M 128 tokens, N 128 tokens, K dk
//   qs      = q [S hi | S lo]   M 128, N 64 + 64, K dk
//   kv      = k^T [wv hi | wv lo (+ lo2)]  M dk, N 64 + 64, K 128 tokens
//   pv      = P hi v + P lo v   M 128, N 64, K 128, P in tensor memory
// Two bf16 terms carry 16 significant bits, so an output is off by about 2^-17
// of its terms before its own rounding (one term would cost as much as that
// rounding again); a state that is returned, in fp32, takes three.  fp16
// terms are scaled by a power of two (per row of P, per block of wv, per S),
// undone on the fp32 result, which keeps them in fp16's range: two are 22 bits.
//
// One block of threads per SM and 64 value columns of a head (dv = 128: two
// blocks share a head, as a cluster when the norm needs the sum over both),
// walking its parts' blocks of 128 tokens.  24 warps, each group one step of the
// pipeline, joined by mbarriers:
//   0-3   scores -> decayed, masked P (a thread has a row)
//   4-7   the decay sums; wv terms; zeros behind the last token
//   8-15  outputs: qs and pv joined, norm, gate (a thread has half a row)
//   16-19 the state: fp32 in registers (a thread has a row of 64 columns, or a
//         half row), S <- a S + kv, and its terms for the next block's qs
//   20    loads of k and v (TMA, 128-byte swizzled tiles of 128 rows x 64 columns)
//   21    issues the products
//   22,23 loads of q; loads of z and stores of the outputs
// The products of a block are issued scores, kv, qs, pv: while the P warps turn
// block c's scores around and the output warps still read block c - 1's qs and
// pv, the tensor cores do its kv.
// The loops are kept rolled where registers allow: unrolled, the instruction
// streams of the groups outgrew the instruction caches (half of all stalls).
// The summaries' kernel (kSum) is the part of it that makes kv and the state: 14
// warps, two threads a row, two wv tiles and kv accumulators in turn.
//
// Bound by the chain scores -> P -> pv -> outputs of a block and the state's kv ->
// S -> qs beside it, each link a wait of 120-200 cycles and a pass of exponentials
// or roundings by one or two warps a scheduler: a block of 128 tokens takes 3.0 to
// 3.4 us for dk = dv = 64 and 4.5 us for 128 (3.6 and 4.4 with every SM busy), of
// which the tensor cores are busy 0.7 and 1.1.  A thread of the outputs kernel
// spills 56 to 112 bytes of registers.  Measured: 16384 tokens, 6 heads of 64, fp16,
// gated (one wave, cold caches): summaries 18 us, scan 7.6, outputs 34, 50 us a
// call, 1.3 TB/s of the call's 63 MB; 65536 tokens, 4 heads of 128, bf16: 49 + 8.8 +
// 145, 188 to 195 us a call, 1.8 TB/s of 336 MB; 28 prompts of 4 to 7442 tokens, 16
// heads of 128: 71 + 7.5 + 172, 255 us.
#pragma once
#include "hla_common.cuh"
#include "tc_ptx.cuh"

namespace gtr {
namespace hla {

using tc::saddr;

constexpr int kTile = kC * 128;          // 128 rows x 64 16-bit columns: 16 KB
constexpr int kTcThreads = 24 * 32;
constexpr int kSumThreads = 14 * 32;

struct Maps {
  CUtensorMap q, k, v, z, o;
};

template <typename T, int DK, bool kSum> struct Layout {
  static constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  static constexpr int kTerms = kBf16 ? 3 : 2;       // of wv
  static constexpr int kQTile = DK / 64 * kTile;
  static constexpr int kNQ = kSum ? 0 : DK == 64 ? 2 : 1;   // stages: q of the next block comes from L2 for dk = 128
  static constexpr int kNK = kSum && DK == 64 ? 3 : 2;
  static constexpr int kNV = kNK;
  static constexpr int kNW = kSum ? 2 : 1;            // wv tiles, and kv accumulators
  static constexpr int kNZ = DK == 64 ? 2 : 1;
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + kNQ * kQTile;
  static constexpr int kV = kK + kNK * kQTile;
  static constexpr int kW = kV + kNV * kTile;
  static constexpr int kWTile = kTerms * kTile;
  static constexpr int kS = kW + kNW * kWTile;        // S hi, S lo: dk rows x 64 columns each
  static constexpr int kSTile = DK * 128;
  static constexpr int kZ = kS + (kSum ? 0 : 2 * kSTile);   // z, then the outputs over it
  static constexpr int kG = kZ + (kSum ? 0 : kNZ * kTile);         // [2][128] log2-decays l, then G
  static constexpr int kU = kG + 2 * kC * 4;          // [2][128] e^{G_b - G_j}
  static constexpr int kX = kU + 2 * kC * 4;          // [128] the other half's sums of squares
  static constexpr int kRms = kX + kC * 4;            // [64] the norm's weights
  static constexpr int kMisc = kRms + 64 * 4;         // [2][4] sums of l over 32 tokens; the tensor memory address before them
  static constexpr int kBars = kMisc + 32;
  // mbarriers, as indexes
  static constexpr int kQF = 0, kQE = kQF + kNQ, kKF = kQE + kNQ, kKE = kKF + kNK, kVF = kKE + kNK, kVE = kVF + kNV;
  static constexpr int kZF = kVE + kNV, kOS = kZF + kNZ, kScF = kOS + kNZ, kPF = kScF + 1, kPvF = kPF + 1;
  static constexpr int kOE = kPvF + 1, kSF = kOE + 1, kSE = kSF + 1, kWF = kSE + 1, kWE = kWF + kNW;
  static constexpr int kKvF = kWE + kNW, kKvE = kKvF + kNW, kGF = kKvE + kNW, kGE = kGF + 2, kXF = kGE + 2, kXE = kXF + 1;
  static constexpr int kNumBars = kXE + 1;
  // fp16 only: exponents of P [2][128], one byte each, of wv [4] and S [2]; maxima of the builders [8] and of S [4]
  static constexpr int kPExp = kBars + kNumBars * 8;
  static constexpr int kExp = kPExp + (kBf16 ? 0 : 2 * kC);
  static constexpr int kSmem = kExp + (kBf16 ? 0 : 72);
  static_assert(kSmem <= 232448, "shared memory of one block");
};

// Tensor memory columns (512)
constexpr uint32_t kTmSc = 0;      // scores, then P hi in [0, 64)
constexpr uint32_t kTmPlo = 128;   // P lo
constexpr uint32_t kTmQS = 192;    // q S hi | q S lo
constexpr uint32_t kTmPV = 320;
constexpr uint32_t kTmKV = 384;    // kv hi | kv lo

// Instruction descriptor, kind::f16, fp32 accumulation
__host__ __device__ constexpr uint32_t idesc(bool bf16, int a_mn, int b_mn, int m, int n) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(saddr(dst)), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(saddr(bar))
      : "memory");
}
// Shared -> global, as part of the thread's bulk group; no coordinate is negative, c0 is a multiple of 64 elements.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
               "r"(c0), "r"(c1), "r"(c2), "r"(saddr(src))
               : "memory");
}
// A line of global memory into L2.
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* map, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map), "r"(c0), "r"(c1),
               "r"(c2)
               : "memory");
}

// 32 lanes x 32 bit, N columns (thread t of warp w <- lane 32 (w % 4) + t); use after ld_wait
__device__ __forceinline__ void tm_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tm_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
// 16 lanes x 32 bit in two halves of 16 columns (the M = 64 accumulator: row r in lane 32 (r / 16) + r % 16)
__device__ __forceinline__ void tm_ld16x2(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16], 16;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// Waits for this thread's loads; the registers are operands, so that no use of them is scheduled before it.
template <int N> __device__ __forceinline__ void tm_wait(uint32_t (&r)[N]) {
  static_assert(N == 8 || N == 16 || N == 32, "");
  if constexpr (N == 8)
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
                 : "memory");
  else if constexpr (N == 16)
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15])
                 :
                 : "memory");
  else
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

// Two fp32 in one 64-bit register (add / mul / fma .f32x2: one issue for two)
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t pack2(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint64_t both(float a) { return tc::f2pack(a, a); }

// The registers of a thread of a warp group, out of the kLaunchRegs it was launched with.
constexpr int kLaunchRegs = 80;    // 65536 / 768, a multiple of 8
template <int N> __device__ __forceinline__ void set_registers() {
  static_assert(N % 8 == 0 && N >= 24 && N <= 256, "");
  if constexpr (N > kLaunchRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  if constexpr (N < kLaunchRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// Shares of the six warp groups (the state is 64 registers of a thread for dk
// = 128, 32 for dk = 64).
template <int DK> struct Regs {
  static constexpr int kP = DK == 128 ? 56 : 64, kBuild = kP, kOut = DK == 128 ? 88 : 96;
  static constexpr int kState = DK == 128 ? 128 : 80, kMisc = DK == 128 ? 64 : 80;
  static_assert(kP + kBuild + 2 * kOut + kState + kMisc <= 6 * kLaunchRegs, "no more than the block was launched with");
};

__device__ __forceinline__ void tm_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

template <typename T> struct T2;
template <> struct T2<__half> {
  using t = __half2;
  static __device__ __forceinline__ t from(float a, float b) { return __floats2half2_rn(a, b); }
  static __device__ __forceinline__ float2 to(t x) { return __half22float2(x); }
};
template <> struct T2<__nv_bfloat16> {
  using t = __nv_bfloat162;
  static __device__ __forceinline__ t from(float a, float b) { return __floats2bfloat162_rn(a, b); }
  static __device__ __forceinline__ float2 to(t x) { return __bfloat1622float2(x); }
};
template <typename T> __device__ __forceinline__ uint32_t word(typename T2<T>::t x) {
  uint32_t u;
  memcpy(&u, &x, 4);
  return u;
}
// two 16-bit values as two fp32
template <typename T> __device__ __forceinline__ uint64_t widen(uint32_t u) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) return pack2(u << 16, u & 0xffff0000u);
  typename T2<T>::t x;
  memcpy(&x, &u, 4);
  const float2 f = T2<T>::to(x);
  return tc::f2pack(f.x, f.y);
}
template <typename T> __device__ __forceinline__ uint32_t narrow(uint64_t x) {
  const float2 f = tc::f2unpack(x);
  return word<T>(T2<T>::from(f.x, f.y));
}
// The rounding of x to T; x becomes what is left.
template <typename T> __device__ __forceinline__ uint32_t term(uint64_t& x) {
  const uint32_t h = narrow<T>(x);
  x = tc::ffma2(widen<T>(h), both(-1.f), x);
  return h;
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// One lane of the (whole) warp, the same each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t a, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
// Four bytes into the other block's shared memory, counted on its barrier as they land.
__device__ __forceinline__ void peer_send(uint32_t a, float v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(a),
               "r"(__float_as_uint(v)), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void peer_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Bounded waits, short in code (there are some 35 of them): a probe that fails
// has slept for at most 20 us, so kProbes of them, a second or so as they are
// seen here and 20 s at the very most, end any wait.
constexpr uint32_t kProbes = 1u << 20;
// `ok` false: one probe, no more.
__device__ __forceinline__ void probe(uint64_t* b, uint32_t parity, bool& ok) {
  uint32_t n = ok ? kProbes : 0;
#pragma unroll 1
  while (!tc::mbar_try(b, parity)) {
    if (n == 0) {
      ok = false;
      return;
    }
    --n;
  }
}
// The same, acquiring what the other block of the cluster released.
__device__ __forceinline__ void cluster_wait(uint64_t* b, uint32_t parity, bool& ok) {
  uint32_t n = ok ? kProbes : 0;
#pragma unroll 1
  while (true) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(saddr(b)), "r"(parity), "r"(20000u)
        : "memory");
    if (done) return;
    if (n == 0) {
      ok = false;
      return;
    }
    --n;
  }
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One thread's columns of a state tile of dk rows x 64: M = 128 accumulators
// give a thread a whole row, M = 64 ones two runs of 16 columns (32 apart).
template <int DK> struct StateCols {
  static constexpr int kN = DK == 128 ? 64 : 32;
  // row, and first column of the 16-column run e
  static __device__ __forceinline__ int row(int warp4, int lane) {
    return DK == 128 ? warp4 * 32 + lane : warp4 * 16 + (lane & 15);
  }
  static __device__ __forceinline__ int col(int run, int lane) {
    return DK == 128 ? run * 16 : run * 32 + (lane >> 4) * 16;
  }
};

// kGated: with the norm and the gate.  kPair: the two halves of dv = 128 with a
// norm, as a cluster of two.
template <typename T, int DK, bool kSum, bool kGated, bool kPair>
__global__ void __launch_bounds__(kSum ? kSumThreads : kTcThreads, 1) hla_tc(const Params p,
                                                                             const __grid_constant__ Maps maps,
                                                                             const int halves) {
  using L = Layout<T, DK, kSum>;
  constexpr bool kBf16 = L::kBf16;
  extern __shared__ __align__(1024) uint8_t tiles[];
  uint8_t* sm = tiles;
  float* Ls = reinterpret_cast<float*>(sm + L::kG);
  float* Us = reinterpret_cast<float*>(sm + L::kU);
  float* Xs = reinterpret_cast<float*>(sm + L::kX);
  float* rmsw = reinterpret_cast<float*>(sm + L::kRms);
  float* wsum = reinterpret_cast<float*>(sm + L::kMisc);           // [2][4], of a block like Ls and Us
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::kMisc);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::kBars);
  int8_t* pexp = reinterpret_cast<int8_t*>(sm + L::kPExp);          // fp16 only, as the next three
  int* ew = reinterpret_cast<int*>(sm + L::kExp);
  int* es = ew + 4;
  float* wmax = reinterpret_cast<float*>(ew + 6);                   // [8] builders, [4] state
  constexpr int kQF = L::kQF, kQE = L::kQE, kKF = L::kKF, kKE = L::kKE, kVF = L::kVF, kVE = L::kVE, kZF = L::kZF;
  constexpr int kOS = L::kOS, kScF = L::kScF, kPF = L::kPF, kPvF = L::kPvF, kOE = L::kOE, kSF = L::kSF, kSE = L::kSE;
  constexpr int kWF = L::kWF, kWE = L::kWE, kKvF = L::kKvF, kKvE = L::kKvE, kGF = L::kGF, kGE = L::kGE, kXF = L::kXF;
  constexpr int kXE = L::kXE;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // roles: the summary has no score and output warps
  enum { kP = 0, kBuild = 1, kOut = 2, kState = 3, kLoad = 4, kMma = 5, kLoadQ = 6, kLoadZ = 7 };
  const int role = kSum ? (warp < 8 ? kBuild : warp < 12 ? kState : warp - 8) : (warp < 8 ? warp >> 2 : warp < 16 ? kOut : warp < 20 ? kState : warp - 16);
  if ((saddr(sm) & 1023u) != 0u) {
    if (tid == 0) gtr_flag(kStatusBadShape);
    return;
  }
  if (tid < L::kNumBars) {
    // arrivals: one (a copy's issue, a product's commit), or one of each warp of the group
    const int i = tid;
    const bool out = i == kOE || (i >= kOS && i < kOS + L::kNZ);
    const bool wf = i >= kWF && i < kWF + L::kNW, readers = i >= kGE && i < kGE + 2;
    const bool four = i == kPF || wf || i == kSF || (i >= kKvE && i < kKvE + L::kNW) || (i >= kGF && i < kGF + 2);
    tc::mbar_init(bar + i, out || (kSum && wf) ? 8 : four ? 4 : readers ? (kSum ? 4 : 16) : i == kXE ? kC : 1);
    tc::mbar_fence_init();
  }
  if (role == kMma) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  tc::tc_before_sync();
  __syncthreads();
  tc::tc_after_sync();
  if constexpr (kPair) cluster_sync();
  pdl_wait();
  pdl_trigger();
  const uint32_t tm = *tmem_slot;
  const int half = (int)blockIdx.x % halves, group_j = (int)blockIdx.x / halves;
  Range rg;
  locate<kC>(p, group_j, reinterpret_cast<int*>(Ls), rg);
  if (kGated && tid < 64) rmsw[tid] = p.w ? __ldg(p.w + half * 64 + tid) : 1.f;
  __syncthreads();                                             // the scratch becomes the decays
  Part cut;                                                    // the summary's one part
  bool has_cut = false;
  if constexpr (kSum) {
    has_cut = cut_part<kC>(p, rg, cut);
    if (!has_cut && tid == 0 && half == 0) p.chains[group_j] = Chain{0, 0, 0, 0};
  }
  const int w4 = warp & 3, row = w4 * 32 + lane;               // a token row, or a lane of an accumulator
  const uint32_t lane_base = (uint32_t)(w4 * 32) << 16;
  const int share = p.H / p.Hk;                                // heads of a key head
  uint32_t it = 0;                                             // blocks of tokens since the start
  uint32_t is = 0;                                             // those that had a state before them
  // Bounded waits: a failed probe returns at the latest after 20 us, so kProbes of them end in any case.  A thread
  // whose wait ran out (ok false) probes once where it waited, arrives nowhere and issues nothing, but walks on: what it
  // reads and writes stays in bounds whatever the order, and the barriers of its group (bar.sync, which has no limit)
  // still get it.  So every role comes to its end.
  bool ok = true;
  auto wait = [&](int b, uint32_t parity) { probe(bar + b, parity, ok); };
  // two barriers: their first probes are in flight together (a probe takes about 120 cycles)
  auto wait2 = [&](int b, uint32_t pb, int c, uint32_t pc) {
    const uint32_t x = tc::mbar_try(bar + b, pb), y = tc::mbar_try(bar + c, pc);
    if (!x) wait(b, pb);
    if (!y) wait(c, pc);
  };
  // one arrival for a warp, after all its lanes
  auto warp_arrive = [&](int b) {
    __syncwarp();
    if (lane == 0 && ok) tc::mbar_arrive_one(bar + b);
  };
  auto for_parts = [&](auto&& body, auto flag) {
    if constexpr (kSum) {
      if (has_cut) body(cut);
    } else {
      Part g;
      Walk walk{rg.a, rg.x1 - rg.x0};
      while (next_part<kC, decltype(flag)::value>(p, walk, g)) body(g);
    }
  };
  constexpr std::true_type kRecord{};                          // the role that records bad slots
  constexpr std::false_type kQuiet{};
  // the state after the part is needed / there is one before it
  auto wants_end = [&](const Part& g) { return kSum || (g.last && p.state_out); };
  auto has_start = [&](const Part& g) { return !kSum && (!g.first || g.start); };

  if (role == kLoad) {
    if constexpr (!kSum) set_registers<Regs<DK>::kMisc>();
    for_parts([&](const Part& g) {
      const int hk = g.h / share;
      if (lane == 0) {
        for (int c = 0; c < g.nb && ok; ++c) {
          const uint32_t i = it + c;
          const int t = g.t0 + c * kC;
          const int sk = i % L::kNK, sv = i % L::kNV;
          wait(kKE + sk, (i / L::kNK & 1) ^ 1);
          if (!ok) break;
          tc::mbar_arrive_tx(bar + kKF + sk, L::kQTile);
          for (int x = 0; x < DK / 64; ++x)
            tma_load_3d(sm + L::kK + sk * L::kQTile + x * kTile, &maps.k, x * 64, hk, t, bar + kKF + sk);
          wait(kVE + sv, (i / L::kNV & 1) ^ 1);
          if (!ok) break;
          tc::mbar_arrive_tx(bar + kVF + sv, kTile);
          tma_load_3d(sm + L::kV + sv * kTile, &maps.v, half * 64, g.h, t, bar + kVF + sv);
        }
      }
      it += g.nb;
    }, kRecord);
  } else if (role == kMma) {
    if constexpr (!kSum) set_registers<Regs<DK>::kMisc>();
    const bool lead = elect_one();
    for_parts([&](const Part& g) {
      constexpr uint32_t kIdSc = idesc(kBf16, 0, 0, 128, 128), kIdQS = idesc(kBf16, 0, 1, 128, 128);
      constexpr uint32_t kIdKV = idesc(kBf16, 1, 1, DK, 128), kIdKV3 = idesc(kBf16, 1, 1, DK, 64);
      constexpr uint32_t kIdPV = idesc(kBf16, 0, 1, 128, 64);
      // the same in every lane; the reduction says so to the compiler
      const int nb = (int)__reduce_max_sync(0xffffffffu, (unsigned)g.nb);
      const bool want_end = wants_end(g);
      const int terms = want_end ? L::kTerms : 2;
      for (int c = 0; c < nb; ++c) {
        const uint32_t i = it + c, par = i & 1;
        const int sk = i % L::kNK, sv = i % L::kNV;
        const uint8_t* K = sm + L::kK + sk * L::kQTile;
        const uint8_t* V = sm + L::kV + sv * kTile;
        const int sw = i % L::kNW;                               // wv tile and kv accumulator
        const uint32_t pw = i / L::kNW & 1, kv = tm + kTmKV - 128 * sw;
        const uint8_t* W = sm + L::kW + sw * L::kWTile;
        if constexpr (!kSum) {
          const int sq = i % L::kNQ;
          const uint8_t* Q = sm + L::kQ + sq * L::kQTile;
          wait2(kKF + sk, i / L::kNK & 1, kQF + sq, i / L::kNQ & 1);
          tc::tc_after_sync();
          const uint64_t aq = tc::sdesc(saddr(Q), 16, 1024), bk = tc::sdesc(saddr(K), 16, 1024);
          if (lead && ok) {
#pragma unroll
            for (int s = 0; s < DK / 16; ++s) {
              const uint64_t o = (uint64_t)((s >> 2) * (kTile >> 4) + (s & 3) * tc::kStepK);
              tc::mma_f16(tm + kTmSc, aq + o, bk + o, kIdSc, s > 0);
            }
            tc::mma_commit(bar + kScF);
          }
          __syncwarp();
        } else {
          wait(kKF + sk, i / L::kNK & 1);
        }
        wait2(kWF + sw, pw, kKvE + sw, pw ^ 1);
        tc::tc_after_sync();
        if ((c + 1 < nb || want_end) && lead && ok) {
          const uint64_t ak = tc::sdesc(saddr(K), kTile, 1024), bw = tc::sdesc(saddr(W), kTile, 1024);
#pragma unroll 1
          for (int s = 0; s < kC / 16; ++s)
            tc::mma_f16(kv, ak + s * tc::kStepMN, bw + s * tc::kStepMN, kIdKV, s > 0);
          if (L::kTerms == 3 && terms == 3) {
            const uint64_t bw3 = tc::sdesc(saddr(W + 2 * kTile), kTile, 1024);
#pragma unroll 1
            for (int s = 0; s < kC / 16; ++s)
              tc::mma_f16(kv + 64, ak + s * tc::kStepMN, bw3 + s * tc::kStepMN, kIdKV3, 1u);
          }
        }
        if (lead && ok) {
          tc::mma_commit(bar + kKvF + sw);
          tc::mma_commit(bar + kWE + sw);
          tc::mma_commit(bar + kKE + sk);
        }
        __syncwarp();
        if constexpr (!kSum) {
          const int sq = i % L::kNQ;
          const uint64_t aq = tc::sdesc(saddr(sm + L::kQ + sq * L::kQTile), 16, 1024);
          // the terms of S; qs and pv of the block before are read
          const bool state = c > 0 || has_start(g);
          if (state) wait2(kSF, is & 1, kOE, par ^ 1);
          else wait(kOE, par ^ 1);
          tc::tc_after_sync();
          if (state) {
            const uint64_t bs = tc::sdesc(saddr(sm + L::kS), L::kSTile, 1024);
            if (lead && ok) {
#pragma unroll 1
              for (int s = 0; s < DK / 16; ++s) {
                const uint64_t o = (uint64_t)((s >> 2) * (kTile >> 4) + (s & 3) * tc::kStepK);
                tc::mma_f16(tm + kTmQS, aq + o, bs + s * tc::kStepMN, kIdQS, s > 0);
              }
              tc::mma_commit(bar + kSE);
            }
            ++is;
          }
          if (lead && ok) tc::mma_commit(bar + kQE + sq);
          __syncwarp();
          wait(kPF, par);
          tc::tc_after_sync();
          const uint64_t bv = tc::sdesc(saddr(V), kTile, 1024);
          if (lead && ok) {
#pragma unroll 1
            for (int s = 0; s < kC / 16; ++s)
              tc::mma_f16_ts(tm + kTmPV, tm + kTmSc + 8 * s, bv + s * tc::kStepMN, kIdPV, s > 0);
#pragma unroll 1
            for (int s = 0; s < kC / 16; ++s)
              tc::mma_f16_ts(tm + kTmPV, tm + kTmPlo + 8 * s, bv + s * tc::kStepMN, kIdPV, 1u);
            tc::mma_commit(bar + kPvF);
          }
        }
        if (lead && ok) tc::mma_commit(bar + kVE + sv);
        __syncwarp();
      }
      it += nb;
    }, kQuiet);
    if (it > 0) {
      // the last arrival a product makes on this memory
      const uint32_t i = it - 1;
      wait(kVE + i % L::kNV, i / L::kNV & 1);
    }
  } else if (role == kBuild) {
    if constexpr (!kSum) set_registers<Regs<DK>::kBuild>();
    // the summary, where nothing else hides it: two threads a row
    constexpr int kSubs = kSum ? 2 : 1, kUnits = 8 / kSubs;
    const int sub = kSum ? warp >> 2 : 0, u0 = sub * kUnits;
    for_parts([&](const Part& g) {
      const bool want_end = wants_end(g);
      // a block ahead, and turned when it is used (rows past the end read the last one)
      float raw = g.len > 0 ? load_g(p, g.t0 + min(row, g.len - 1), g.h) : 0.f;
      for (int c = 0; c < g.nb; ++c) {
        const uint32_t i = it + c;
        const int nv = min(kC, g.len - c * kC);                  // tokens of this block
        const float lc = row < nv ? log2_decay(raw) : 0.f;
        if (c + 1 < g.nb) raw = load_g(p, g.t0 + min((c + 1) * kC + row, g.len - 1), g.h);
        // the sums from the back: all 32 in lane 0, then without the token itself
        float suf = lc;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const float b = __shfl_down_sync(0xffffffffu, suf, d);
          if (lane + d < 32) suf += b;
        }
        const float all = suf, behind = __shfl_down_sync(0xffffffffu, suf, 1);
        suf = lane == 31 ? 0.f : behind;
        if (sub == 0) {
          wait(kGE + (i & 1), (i >> 1 & 1) ^ 1);
          Ls[(i & 1) * kC + row] = lc;
          Us[(i & 1) * kC + row] = tc::ex2(suf);
          if (lane == 0) wsum[(i & 1) * 4 + w4] = all;
          warp_arrive(kGF + (i & 1));
        }
        tc::named_barrier(1, 128 * kSubs);
        const float* ws = wsum + (i & 1) * 4;
        float R = suf;
#pragma unroll
        for (int x = 1; x < 4; ++x)
          if (x > w4) R += ws[x];
        const int sv = i % L::kNV, sk = i % L::kNK;
        wait(kVF + sv, i / L::kNV & 1);
        uint8_t* V = sm + L::kV + sv * kTile + row * 128;
        const bool build = c + 1 < g.nb || want_end;
        const bool live = row < nv;
        const float w = tc::ex2(R);
        // this row's unit u of v; nothing of others' data behind the last token (maybe NaN)
        auto unit = [&](int u) {
          const uint4 x = *reinterpret_cast<const uint4*>(V + ((u ^ (row & 7)) << 4));
          return live ? x : make_uint4(0, 0, 0, 0);
        };
        float up = 1.f;
        int exp_w = 0;
        if (!kBf16 && build) {
          // a power of two that brings the block's largest |w v| under 2^15
          uint32_t mx = 0;                                       // |fp16| orders as its bits, NaN on top
#pragma unroll 1
          for (int u = u0; u < u0 + kUnits; ++u) {
            const uint4 v = unit(u);
            const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) mx = __vmaxu2(mx, x[e] & 0x7fff7fffu);
          }
          const float2 f = tc::f2unpack(widen<T>(mx));
          const float m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(f.x, f.y) * w)));
          if (lane == 0) wmax[4 * sub + w4] = m;
          tc::named_barrier(1, 128 * kSubs);
          float top = 0.f;
#pragma unroll
          for (int x = 0; x < 4 * kSubs; ++x) top = fmaxf(top, wmax[x]);
          exp_w = tc::scale_exp(top);
          up = tc::pow2i(exp_w);
        }
        const int sw = i % L::kNW;
        wait(kWE + sw, (i / L::kNW & 1) ^ 1);
        if (build) {
          // the tile's last product is done; the exponent of four blocks ago, in this slot, is long read
          if (!kBf16 && row == 0 && sub == 0) ew[i & 3] = exp_w;
          uint8_t* W = sm + L::kW + sw * L::kWTile + row * 128;
          const uint64_t f = both(w * up);
#pragma unroll 1
          for (int u = u0; u < u0 + kUnits; ++u) {
            const uint4 v = unit(u);
            const uint32_t x[4] = {v.x, v.y, v.z, v.w};
            uint32_t t[L::kTerms][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint64_t y = tc::fmul2(widen<T>(x[e]), f);
#pragma unroll
              for (int n = 0; n + 1 < L::kTerms; ++n) t[n][e] = term<T>(y);
              t[L::kTerms - 1][e] = narrow<T>(y);
            }
            const int off = (u ^ (row & 7)) << 4;
#pragma unroll
            for (int n = 0; n < L::kTerms; ++n)
              if (n < 2 || want_end)
                *reinterpret_cast<uint4*>(W + n * kTile + off) = make_uint4(t[n][0], t[n][1], t[n][2], t[n][3]);
          }
        }
        if (nv < kC) {
          // rows behind the sequence's last token hold others' data: zeros, so
          // that nothing of them (a NaN times a zero weight) enters a product
          wait(kKF + sk, i / L::kNK & 1);
          if (!live) {
            uint8_t* K = sm + L::kK + sk * L::kQTile + row * 128;
            const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int u = u0; u < u0 + kUnits; ++u) {
              // (any unit's place in the row: all of them are zeroed, by one of the two threads)
              *reinterpret_cast<uint4*>(V + ((u ^ (row & 7)) << 4)) = zero;
#pragma unroll
              for (int x = 0; x < DK / 64; ++x) *reinterpret_cast<uint4*>(K + x * kTile + ((u ^ (row & 7)) << 4)) = zero;
            }
          }
        }
        tc::fence_async_smem();
        warp_arrive(kWF + sw);
      }
      it += g.nb;
    }, kQuiet);
  } else if (role == kState) {
    if constexpr (!kSum) set_registers<Regs<DK>::kState>();
    using SC = StateCols<DK>;
    constexpr int kRuns = SC::kN / 16;
    const int r = SC::row(w4, lane);
    uint64_t S[SC::kN / 2];                                       // two columns each
    // S in two terms as the operand of the next block's qs
    auto put = [&]() {
      uint64_t up = both(1.f);
      int exp_s = 0;
      if (!kBf16) {
        uint32_t mx = 0;
#pragma unroll
        for (int e = 0; e < SC::kN / 2; ++e) {
          const float2 f = tc::f2unpack(S[e]);
          mx = max(mx, max(__float_as_uint(f.x) & 0x7fffffffu, __float_as_uint(f.y) & 0x7fffffffu));
        }
        const float m = __uint_as_float(__reduce_max_sync(0xffffffffu, mx));
        if (lane == 0) wmax[8 + w4] = m;
        tc::named_barrier(2, 128);
        const int e = tc::scale_exp(fmaxf(fmaxf(wmax[8], wmax[9]), fmaxf(wmax[10], wmax[11])));
        tc::named_barrier(2, 128);                               // read before the next block's are written
        up = both(tc::pow2i(e));
        exp_s = e;
      }
      wait(kSE, (is & 1) ^ 1);
      // the product of the state before is done, and was issued after the outputs had taken the exponent of the
      // one before that (kOE), which this overwrites
      if (!kBf16 && w4 == 0 && lane == 0) es[is & 1] = exp_s;
      ++is;
      uint8_t* D = sm + L::kS + r * 128;
#pragma unroll
      for (int x = 0; x < kRuns; ++x) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint64_t a = S[8 * x + 4 * b + e];
            if (!kBf16) a = tc::fmul2(a, up);
            hi[e] = term<T>(a);
            lo[e] = narrow<T>(a);
          }
          const int off = ((SC::col(x, lane) / 8 + b) ^ (r & 7)) << 4;
          *reinterpret_cast<uint4*>(D + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(D + L::kSTile + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      tc::fence_async_smem();
      warp_arrive(kSF);
    };
    const size_t hs = (size_t)DK * p.dv, at = (size_t)r * p.dv + half * 64;
    auto run = [&](const Part& g) {
      const bool want_end = wants_end(g);
      const float* src = kSum ? nullptr : start_state(p, g, group_j);
#pragma unroll
      for (int x = 0; x < kRuns; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 f = src ? *reinterpret_cast<const float4*>(src + at + SC::col(x, lane) + 4 * e)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
          S[8 * x + 2 * e] = tc::f2pack(f.x, f.y);
          S[8 * x + 2 * e + 1] = tc::f2pack(f.z, f.w);
        }
      float total = 0.f;
      // c = -1: the terms of the state before the first block
      for (int c = has_start(g) ? -1 : 0; c < g.nb; ++c) {
        if (c >= 0) {
          const uint32_t i = it + c;
          const int sw = i % L::kNW;
          const uint32_t kv = tm + lane_base + kTmKV - 128 * sw;
          wait2(kGF + (i & 1), i >> 1 & 1, kKvF + sw, i / L::kNW & 1);
          const float4 ws = *reinterpret_cast<const float4*>(wsum + (i & 1) * 4);
          const float la = (ws.x + ws.y) + (ws.z + ws.w);
          warp_arrive(kGE + (i & 1));
          tc::tc_after_sync();
          if (c + 1 < g.nb || want_end) {
            total += la;
            const uint64_t a = both(tc::ex2(la));
            const uint64_t down = both(kBf16 ? 1.f : tc::pow2i(-ew[i & 3]));
#pragma unroll
            for (int x = 0; x < kRuns; ++x) {
              uint32_t hi[16], lo[16];
              if constexpr (DK == 128) {
                tm_ld16(kv + 16 * x, hi);
                tm_ld16(kv + 64 + 16 * x, lo);
              } else {
                tm_ld16x2(kv + 32 * x, hi);
                tm_ld16x2(kv + 64 + 32 * x, lo);
              }
              tm_wait(hi);
              tm_wait(lo);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                uint64_t d = add2(pack2(hi[2 * e], hi[2 * e + 1]), pack2(lo[2 * e], lo[2 * e + 1]));
                if (!kBf16) d = tc::fmul2(d, down);
                S[8 * x + e] = tc::ffma2(a, S[8 * x + e], d);
              }
            }
          }
          tc::tc_before_sync();
          warp_arrive(kKvE + sw);
        }
        if (!kSum && c + 1 < g.nb) put();
      }
      it += g.nb;
      if (want_end) {
        float* dst = kSum ? p.wsS + (size_t)group_j * hs : p.state_out + ((size_t)g.slot * p.H + g.h) * hs;
#pragma unroll
        for (int x = 0; x < kRuns; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 a = tc::f2unpack(S[8 * x + 2 * e]), b = tc::f2unpack(S[8 * x + 2 * e + 1]);
            *reinterpret_cast<float4*>(dst + at + SC::col(x, lane) + 4 * e) = make_float4(a.x, a.y, b.x, b.y);
          }
        if (kSum && half == 0 && w4 == 0 && lane == 0) {
          p.wsA[group_j] = total;
          p.chains[group_j] = chain_of<kC>(p, rg, g, group_j);
        }
      }
    };
    if constexpr (kSum) {
      for_parts(run, kQuiet);
    } else {
      // a part behind: the state the next one starts from is on its way into L2 meanwhile
      Walk walk{rg.a, rg.x1 - rg.x0};
      Part g, n;
      bool have = false;
      while (true) {
        const bool more = next_part<kC>(p, walk, n);
        if (more) {
          const float* src = start_state(p, n, group_j);
          if (src) {
            prefetch_l2(src + at + SC::col(0, lane));
            if (DK == 128) prefetch_l2(src + at + 32);
          }
        }
        if (have) run(g);
        if (!more) break;
        g = n;
        have = true;
      }
    }
  } else if constexpr (!kSum) {
    if (role == kP) {
      set_registers<Regs<DK>::kP>();
      {
        // P lo right of the diagonal is zero for good
        uint32_t zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int b = 2 * w4 + 2; b < 8; ++b) tm_st8(tm + lane_base + kTmPlo + 8 * b, zero);
      }
      for_parts([&](const Part& g) {
        for (int c = 0; c < g.nb; ++c) {
          const uint32_t i = it + c, par = i & 1;
          wait(kGF + (i & 1), i >> 1 & 1);                       // long before the scores
          const float* U = Us + (i & 1) * kC;
          const float* ws = wsum + (i & 1) * 4;
          // sums of l from the start of the row's 16 tokens (pre16) and of its 32 to the row
          float* L_row = Ls + (i & 1) * kC + row;
          const float l = *L_row;
          float pre16 = l;
#pragma unroll
          for (int d = 1; d < 16; d <<= 1) {
            const float y = __shfl_up_sync(0xffffffffu, pre16, d);
            if ((lane & 15) >= d) pre16 += y;
          }
          const float half0 = __shfl_sync(0xffffffffu, pre16, 15);
          const float pre32 = lane < 16 ? pre16 : pre16 + half0;
          // the row's own decay, to the last bit: up to 15 of them make a weight
          const float decay = l > -1.f ? 1.f + expm1_small(l * kLn2) : tc::ex2(l);
          const float past16 = lane < 16 ? 0.f : tc::ex2(pre16);
          // the weights of the last token one, two and three 32s before the row's
          const float sum2 = pre32 + ws[max(w4 - 1, 0)], sum3 = sum2 + ws[max(w4 - 2, 0)];
          const float past32 = tc::ex2(pre32), past64 = tc::ex2(sum2), past96 = tc::ex2(sum3);
          // for the outputs: the sum from the block's start
          *L_row = w4 == 0 ? pre32 : w4 == 1 ? sum2 : w4 == 2 ? sum3 : sum3 + ws[0];
          wait(kScF, par);
          tc::tc_after_sync();
          const uint32_t sc = tm + lane_base + kTmSc, plo = tm + lane_base + kTmPlo;
          float up = 1.f;
          if (!kBf16) {
            // a power of two that brings the row's largest |score| under 2^15
            uint32_t mx = 0;
#pragma unroll 1
            for (int b = 0; b < 2 * w4 + 2; ++b) {
              uint32_t x[16];
              tm_ld16(sc + 16 * b, x);
              tm_wait(x);
              const int diag = 32 * w4 + lane - 16 * b;          // the row's last column of this run
#pragma unroll
              for (int e = 0; e < 16; ++e) mx = max(mx, e <= diag ? x[e] & 0x7fffffffu : 0u);
            }
            const int e = tc::scale_exp(__uint_as_float(mx));
            up = tc::pow2i(e);
            pexp[(i & 1) * kC + row] = (int8_t)e;
          }
          // runs of 16 columns; P hi goes over scores already read (columns
          // [8 b, 8 b + 8) of run b / 2)
#pragma unroll 1
          for (int b = 0; b < 2 * w4; ++b) {
            uint32_t x[16], hi[8], lo[8];
            tm_ld16(sc + 16 * b, x);
            const int back = w4 - (b >> 1);
            const uint64_t f = both((back == 1 ? past32 : back == 2 ? past64 : past96) * up);
            const ulonglong2* u2 = reinterpret_cast<const ulonglong2*>(U + 16 * b);
            tm_wait(x);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const ulonglong2 uj = u2[e];
              uint64_t y = tc::fmul2(pack2(x[4 * e], x[4 * e + 1]), tc::fmul2(uj.x, f));
              hi[2 * e] = term<T>(y);
              lo[2 * e] = narrow<T>(y);
              y = tc::fmul2(pack2(x[4 * e + 2], x[4 * e + 3]), tc::fmul2(uj.y, f));
              hi[2 * e + 1] = term<T>(y);
              lo[2 * e + 1] = narrow<T>(y);
            }
            tm_st8(sc + 8 * b, hi);
            tm_st8(plo + 8 * b, lo);
          }
          // the square on the diagonal
#pragma unroll 1
          for (int b = 2 * w4; b < 2 * w4 + 2; ++b) {
            uint32_t x[16], hi[8], lo[8];
            tm_ld16(sc + 16 * b, x);
            const int diag = 32 * w4 + lane - 16 * b, base = 16 * (b & 1);
            // from the run's last column to the left, one decay a column: rows behind the run start with the weight of
            // that column, rows in it at their own (with zeros until then, or a NaN of a later token)
            float wt[16];
            wt[15] = diag == 15 ? up : base == 0 ? past16 * up : 0.f;
#pragma unroll
            for (int e = 14; e >= 0; --e) {
              const float y = wt[e + 1] * __shfl_sync(0xffffffffu, decay, base + e + 1);
              wt[e] = e == diag ? up : y;
            }
            tm_wait(x);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float m = __uint_as_float(x[e]) * wt[e];
              x[e] = e <= diag ? __float_as_uint(m) : 0u;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              uint64_t z = pack2(x[2 * e], x[2 * e + 1]);
              hi[e] = term<T>(z);
              lo[e] = narrow<T>(z);
            }
            tm_st8(sc + 8 * b, hi);
            tm_st8(plo + 8 * b, lo);
          }
          {
            uint32_t zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 1
            for (int b = 2 * w4 + 2; b < 8; ++b) tm_st8(sc + 8 * b, zero);
          }
          tc::tmem_st_wait();
          tc::tc_before_sync();
          warp_arrive(kPF);
          warp_arrive(kGE + (i & 1));
        }
        it += g.nb;
      }, kQuiet);
    } else if (role == kOut) {
      set_registers<Regs<DK>::kOut>();
      const uint32_t rank = kPair ? blockIdx.x & 1u : 0u;
      const int sub = warp >> 2 & 1;                             // this thread's half of the row: columns 32 sub ..
      const uint32_t pv = tm + lane_base + kTmPV + 32 * sub, qs = tm + lane_base + kTmQS + 32 * sub;
      const ulonglong2* wp = reinterpret_cast<const ulonglong2*>(rmsw + 32 * sub);
      for_parts([&](const Part& g) {
        for (int c = 0; c < g.nb; ++c) {
          const uint32_t i = it + c, par = i & 1;
          const int nv = min(kC, g.len - c * kC);
          const int sz = i % L::kNZ;
          wait2(kZF + sz, i / L::kNZ & 1, kPvF, par);            // z, or the buffer alone
          tc::tc_after_sync();
          const bool state = c > 0 || has_start(g);
          float f1 = p.scale * tc::ex2(Ls[(i & 1) * kC + row]), f2 = p.scale;
          if (!kBf16) {
            f1 *= tc::pow2i(-es[is & 1]);
            f2 *= tc::pow2i(-(int)pexp[(i & 1) * kC + row]);
          }
          const uint64_t f11 = both(f1), f22 = both(f2);
          if (state) ++is;
          // o = qs (hi + lo) and pv joined: 32 columns, two to a register pair
          uint64_t o[16];
          uint64_t ss2 = both(0.f);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t a[8], b[8], d[8];
            tm_ld8(pv + 8 * x, d);
            if (state) {
              tm_ld8(qs + 8 * x, a);
              tm_ld8(qs + 64 + 8 * x, b);
              tm_wait(a);
              tm_wait(b);
            }
            tm_wait(d);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint64_t y = tc::fmul2(f22, pack2(d[2 * e], d[2 * e + 1]));
              if (state)
                y = tc::ffma2(f11, add2(pack2(a[2 * e], a[2 * e + 1]), pack2(b[2 * e], b[2 * e + 1])), y);
              o[4 * x + e] = y;
              ss2 = tc::ffma2(y, y, ss2);
            }
          }
          tc::tc_before_sync();
          warp_arrive(kOE);
          uint8_t* Z = sm + L::kZ + sz * kTile + row * 128;
          auto unit = [&](int u) { return reinterpret_cast<uint4*>(Z + (((4 * sub + u) ^ (row & 7)) << 4)); };
          if constexpr (kGated) {
            const float2 sf = tc::f2unpack(ss2);
            float ss = sf.x + sf.y;
            // this row's entry of U is free (P is done): the two threads' sums meet there
            volatile float* X = Us + (i & 1) * kC + row;
            if (sub == 1) *X = ss;
            tc::named_barrier(3, 256);
            if (sub == 0) {
              ss += *X;
              if constexpr (kPair) {
                // the other half's sum: its copy of ours is free once it has read the block before
                if (row == 0 && ok) tc::mbar_arrive_tx(bar + kXF, kC * 4);
                cluster_wait(bar + kXE, par ^ 1, ok);
                if (ok) peer_send(peer_addr(saddr(Xs + row), rank ^ 1u), ss, peer_addr(saddr(bar + kXF), rank ^ 1u));
              }
            }
            // meanwhile the weight and the gate, without the norm's factor
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const ulonglong2 wa = wp[2 * u], wb = wp[2 * u + 1];
              const uint4 zu = *unit(u);
              const uint32_t zw[4] = {zu.x, zu.y, zu.z, zu.w};
              uint64_t* y = o + 4 * u;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                // z sigmoid(z) = z / (1 + 2^(-z log2 e))
                const uint64_t z = widen<T>(zw[e]);
                const float2 m = tc::f2unpack(tc::fmul2(z, both(-kLog2e)));
                const float2 q = tc::f2unpack(add2(tc::f2pack(tc::ex2(m.x), tc::ex2(m.y)), both(1.f)));
                y[e] = tc::fmul2(y[e], tc::fmul2(z, tc::f2pack(rcp(q.x), rcp(q.y))));
              }
              y[0] = tc::fmul2(y[0], wa.x); y[1] = tc::fmul2(y[1], wa.y);
              y[2] = tc::fmul2(y[2], wb.x); y[3] = tc::fmul2(y[3], wb.y);
            }
            if (sub == 0) {
              if constexpr (kPair) {
                cluster_wait(bar + kXF, par, ok);
                ss += *reinterpret_cast<volatile float*>(Xs + row);
                if (ok) peer_arrive(peer_addr(saddr(bar + kXE), rank ^ 1u));
              }
              *X = rsqrtf(ss / (float)p.dv + kRmsEps);
            }
            tc::named_barrier(3, 256);
            const uint64_t inv2 = both(*X);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = tc::fmul2(o[e], inv2);
          }
          warp_arrive(kGE + (i & 1));
#pragma unroll
          for (int u = 0; u < 4; ++u)
            *unit(u) = make_uint4(narrow<T>(o[4 * u]), narrow<T>(o[4 * u + 1]), narrow<T>(o[4 * u + 2]),
                                  narrow<T>(o[4 * u + 3]));
          if (nv < kC) {
            // behind the sequence's last token the rows are not ours: copied row by row
            tc::named_barrier(3, 256);
            const int t = sub * 128 + row, u = t & 7;
            T* dst = (T*)p.out + (long long)(g.t0 + c * kC) * p.ldo + (long long)g.h * p.dv + half * 64 + u * 8;
            const uint8_t* tile = sm + L::kZ + sz * kTile;
#pragma unroll 1
            for (int r = t >> 3; r < nv; r += 32)
              *reinterpret_cast<uint4*>(dst + r * p.ldo) =
                  *reinterpret_cast<const uint4*>(tile + r * 128 + ((u ^ (r & 7)) << 4));
          }
          tc::fence_async_smem();                               // for the copy engine: the stores, and the next z
          warp_arrive(kOS + sz);
        }
        it += g.nb;
      }, kQuiet);
    } else if (role == kLoadQ) {
      set_registers<Regs<DK>::kMisc>();
      for_parts([&](const Part& g) {
        const int hk = g.h / share;
        if (lane == 0) {
          for (int c = 0; c < g.nb && ok; ++c) {
            const uint32_t i = it + c;
            const int t = g.t0 + c * kC, sq = i % L::kNQ;
            if (L::kNQ == 1)                                     // one buffer: at least from memory into L2
              for (int x = 0; x < DK / 64; ++x) tma_prefetch_3d(&maps.q, x * 64, hk, t);
            wait(kQE + sq, (i / L::kNQ & 1) ^ 1);
            if (!ok) break;
            tc::mbar_arrive_tx(bar + kQF + sq, L::kQTile);
            for (int x = 0; x < DK / 64; ++x)
              tma_load_3d(sm + L::kQ + sq * L::kQTile + x * kTile, &maps.q, x * 64, hk, t, bar + kQF + sq);
          }
        }
        it += g.nb;
      }, kQuiet);
    } else if (role == kLoadZ) {
      // z tiles in, output tiles out: one buffer holds a block's z, then its
      // outputs; it is free once the store has read it
      set_registers<Regs<DK>::kMisc>();
      int pt[L::kNZ] = {}, ph[L::kNZ] = {};                      // the block in each buffer: row (-1: no store), head
      auto finish = [&](uint32_t i, int sz) {
        wait(kOS + sz, i / L::kNZ & 1);
        if (ok && pt[sz] >= 0) {
          tma_store_3d(&maps.o, sm + L::kZ + sz * kTile, half * 64, ph[sz], pt[sz]);
          tc::bulk_commit();
          tc::bulk_wait_read<0>();
        }
      };
      for_parts([&](const Part& g) {
        if (lane == 0) {
          for (int c = 0; c < g.nb && ok; ++c) {
            const uint32_t i = it + c;
            const int t = g.t0 + c * kC;
#pragma unroll
            for (int sz = 0; sz < L::kNZ; ++sz) {
              if (i % L::kNZ != sz) continue;
              if (i >= L::kNZ) finish(i - L::kNZ, sz);
              if (!ok) break;
              pt[sz] = g.len - c * kC >= kC ? t : -1;
              ph[sz] = g.h;
              if constexpr (kGated) {
                tc::mbar_arrive_tx(bar + kZF + sz, kTile);
                tma_load_3d(sm + L::kZ + sz * kTile, &maps.z, half * 64, g.h, t, bar + kZF + sz);
                // one buffer: the next z at least from memory into L2
                if (L::kNZ == 1 && c + 1 < g.nb) tma_prefetch_3d(&maps.z, half * 64, g.h, t + kC);
              } else {
                tc::mbar_arrive_one(bar + kZF + sz);
              }
            }
          }
        }
        it += g.nb;
      }, kQuiet);
      if (lane == 0) {
#pragma unroll
        for (int back = L::kNZ; back > 0; --back) {
          if (it < (uint32_t)back) continue;
          const uint32_t i = it - back;
#pragma unroll
          for (int sz = 0; sz < L::kNZ; ++sz)
            if (i % L::kNZ == sz) finish(i, sz);
        }
        tc::bulk_wait<0>();
      }
    }
  }
  // a bounded wait ran out: loads and products in flight get time to land before the memory is given up
  __syncwarp();
  if (__any_sync(0xffffffffu, !ok)) {
    if (lane == 0) gtr_flag(kStatusMbarTimeout);
    const unsigned long long t0 = tc::globaltimer();
    while (tc::globaltimer() - t0 < 2000000ull) {}
  }
  __syncwarp();
  tc::tc_before_sync();
  __syncthreads();
  if constexpr (kPair) cluster_sync();
  if (role == kMma) tc::tmem_dealloc(tm, 512);
}

}  // namespace hla
}  // namespace gtr
