// hla_simt.cuh -- the fp32 CUDA-core kernels of the head-decay linear
// attention: prompts token by token (every dtype and head dim), and the form
// for single tokens.
#pragma once
#include <string.h>

#include "hla_common.cuh"
#include "tc_ptx.cuh"

namespace gtr {
namespace hla {

constexpr int kSimtThreads = 256;
constexpr int kSimtBatch = 16;     // tokens staged in shared memory per pass: two a warp

__host__ __device__ inline int simt_smem_floats(int dk, int dv, bool sum) {
  return kSimtBatch * (2 + (sum ? 1 : 2) * dk + dv + (sum ? 0 : kSimtThreads));
}

// Four consecutive elements as fp32.
__device__ __forceinline__ float4 ld4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
template <typename T> __device__ __forceinline__ float4 ld4(const T* p) {
  const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
  T e[4];
  memcpy(e, &u, 8);
  return make_float4(Elem<T>::to_f(e[0]), Elem<T>::to_f(e[1]), Elem<T>::to_f(e[2]), Elem<T>::to_f(e[3]));
}

// One batch of tokens of one head on its way from memory to shared memory:
// thread tid has the four-element units tid, tid + 256 of each tensor's rows
// (at most 16 x 128 elements), held in registers while the batch before is
// computed.
template <typename T, bool kSum> struct Batch {
  float4 k[2], q[2], v[2];
  float l;
  __device__ __forceinline__ void load(const Params& p, long long t0, int n, int h, int hk, int lgk, int lgv) {
    const int tid = threadIdx.x;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int e = (tid + x * kSimtThreads) * 4;
      const int tk = e >> lgk, tv = e >> lgv;
      if (tk < n) {
        const long long off = (long long)hk * p.dk + (e & (p.dk - 1));
        k[x] = ld4((const T*)p.k + (t0 + tk) * p.ldk + off);
        if (!kSum) q[x] = ld4((const T*)p.q + (t0 + tk) * p.ldq + off);
      }
      if (tv < n) v[x] = ld4((const T*)p.v + (t0 + tv) * p.ldv + (long long)h * p.dv + (e & (p.dv - 1)));
    }
    if (tid < n) l = load_g(p, (int)(t0 + tid), h);
  }
  // as: a - 1, and a where a is not near one
  __device__ __forceinline__ void put(float* as, float* ks, float* qs, float* vs, int n, int lgk, int lgv, float scale) {
    const int tid = threadIdx.x;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int e = (tid + x * kSimtThreads) * 4;
      if (e >> lgk < n) {
        *reinterpret_cast<float4*>(ks + e) = k[x];
        if (!kSum)
          *reinterpret_cast<float4*>(qs + e) = make_float4(q[x].x * scale, q[x].y * scale, q[x].z * scale, q[x].w * scale);
      }
      if (e >> lgv < n) *reinterpret_cast<float4*>(vs + e) = v[x];
    }
    if (tid < n) {
      const float x = log2_decay(l);
      as[tid] = x;
      as[kSimtBatch + tid] = x > -1.f ? expm1f(x * kLn2) : exp2f(x);
    }
  }
};

// A group's parts by the recurrence itself, the state spread over the block:
// thread tid has column tid % dv and the ROWS rows from (tid / dv) ROWS, so a
// warp reads a token's k and q values as broadcasts.  kSum: the summary of the
// part before the group's cut; else the outputs, and final states.  Bound by the
// serial chain of its tokens (three operations per state element and token in
// fp32, two rows to an instruction: 306 cycles a token at dk = dv = 64, and 4400
// per batch to add up the partial sums and finish the rows), so the tokens are
// split over many short parts.  One block of the outputs is resident per SM at 16
// rows a thread and more (180 registers; 254 at 64 rows).  1600 tokens, 6 heads of
// 64, fp32: summaries 16 us, scan 13.5, outputs 30 (cold caches), 52 us a call; one
// group for a (sequence, head), uncut, would take 415 us.  16-bit heads of 16 and 32
// dims: 16384 tokens, 6 heads, 143 and 193 us a call.
template <typename T, int ROWS, bool kSum>
__global__ void __launch_bounds__(kSimtThreads) hla_simt(const Params p) {
  extern __shared__ __align__(16) float sm[];
  const int dk = p.dk, dv = p.dv, lgk = __ffs(dk) - 1, lgv = __ffs(dv) - 1;
  float* as = sm;                            // [2][batch] log-decays, decays
  float* ks = as + 2 * kSimtBatch;           // [batch][dk]
  float* qs = ks + kSimtBatch * dk;          // [batch][dk], outputs only
  float* vs = qs + (kSum ? 0 : kSimtBatch * dk);   // [batch][dv]
  float* part = vs + kSimtBatch * dv;        // [batch][threads]: partial o, outputs only
  __shared__ int scratch[40];
  pdl_wait();
  pdl_trigger();
  Range rg;
  locate<kSimtBatch>(p, blockIdx.x, scratch, rg);
  Walk walk{rg.a, rg.x1 - rg.x0};
  Part g;
  const int tid = threadIdx.x, j = tid & (dv - 1), r0 = (tid >> lgv) * ROWS, groups = kSimtThreads >> lgv;
  const size_t hs = (size_t)dk * dv;
  float wt[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) wt[c] = !kSum && p.w && (tid & 31) + 32 * c < dv ? __ldg(p.w + (tid & 31) + 32 * c) : 1.f;
  if (kSum && tid == 0 && !cut_part<kSimtBatch>(p, rg, g)) p.chains[blockIdx.x] = Chain{0, 0, 0, 0};
  while (kSum ? cut_part<kSimtBatch>(p, rg, g) : next_part<kSimtBatch, true>(p, walk, g)) {
    const int h = g.h, hk = h / (p.H / p.Hk);
    Batch<T, kSum> b;
    b.load(p, g.t0, min(kSimtBatch, g.len), h, hk, lgk, lgv);
    alignas(8) float S[ROWS];
    const float* src = kSum ? nullptr : start_state(p, g, blockIdx.x);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) S[r] = src ? src[(size_t)(r0 + r) * dv + j] : 0.f;
    float total = 0.f;                       // the part's summed log2-decay
    for (int b0 = 0; b0 < g.len; b0 += kSimtBatch) {
      const int n = min(kSimtBatch, g.len - b0);
      const long long t0 = (long long)g.t0 + b0;
      __syncthreads();
      b.put(as, ks, qs, vs, n, lgk, lgv, p.scale);
      __syncthreads();
      if (b0 + kSimtBatch < g.len) b.load(p, t0 + kSimtBatch, min(kSimtBatch, g.len - b0 - kSimtBatch), h, hk, lgk, lgv);
      // a warp finishes the outputs of tokens warp and warp + 8: their z is on its way meanwhile
      const int lane = tid & 31, warp = tid >> 5;
      float z[2][4];
      if (!kSum && p.z) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int t = warp + 8 * x;
          const T* zrow = (const T*)p.z + (t0 + t) * p.ldz + (long long)h * dv;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (t < n && lane + 32 * c < dv) z[x][c] = ld_f(zrow + lane + 32 * c);
        }
      }
#pragma unroll 1
      for (int t = 0; t < n; ++t) {
        // S <- a S + k v as S + (a - 1) S + k v for a near one: rounding a itself
        // would be the same relative error at every token, 2^-25 a token for as
        // long as the state remembers
        const float l = as[t], a = as[kSimtBatch + t], v = vs[t * dv + j];
        const bool near_one = l > -1.f;
        total += l;
        const float* k = ks + t * dk + r0;
        const float* q = qs + t * dk + r0;
        float sum = 0.f;
        if constexpr (ROWS < 4) {
#pragma unroll
          for (int r = 0; r < ROWS; ++r) {
            S[r] = fmaf(a, S[r], near_one ? fmaf(k[r], v, S[r]) : k[r] * v);
            if (!kSum) sum = fmaf(q[r], S[r], sum);
          }
        } else {
          // two rows to an instruction; the branch is the block's
          const uint64_t a2 = tc::f2pack(a, a), v2 = tc::f2pack(v, v);
          uint64_t o2 = tc::f2pack(0.f, 0.f), p2 = o2;
          uint64_t* S2 = reinterpret_cast<uint64_t*>(S);
#pragma unroll
          for (int r = 0; r < ROWS / 2; r += 2) {
            const ulonglong2 kk = *reinterpret_cast<const ulonglong2*>(k + 2 * r);
            if (near_one) {
              S2[r] = tc::ffma2(a2, S2[r], tc::ffma2(kk.x, v2, S2[r]));
              S2[r + 1] = tc::ffma2(a2, S2[r + 1], tc::ffma2(kk.y, v2, S2[r + 1]));
            } else {
              S2[r] = tc::ffma2(a2, S2[r], tc::fmul2(kk.x, v2));
              S2[r + 1] = tc::ffma2(a2, S2[r + 1], tc::fmul2(kk.y, v2));
            }
            if (!kSum) {
              const ulonglong2 qq = *reinterpret_cast<const ulonglong2*>(q + 2 * r);
              o2 = tc::ffma2(qq.x, S2[r], o2);
              p2 = tc::ffma2(qq.y, S2[r + 1], p2);
            }
          }
          const float2 x = tc::f2unpack(o2), y = tc::f2unpack(p2);
          sum = x.x + x.y + (y.x + y.y);
        }
        if (!kSum) {
          part[t * kSimtThreads + tid] = sum;
        }
      }
      if (!kSum) {
        __syncthreads();
        // the rows' partial sums, then the norm and the gate
        float o[2][4], inv[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int t = min(warp + 8 * x, n - 1);                // past the end: a row again, not stored
          float ss = 0.f;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            o[x][c] = 0.f;
            if (lane + 32 * c < dv) {
              const float* row = part + t * kSimtThreads + lane + 32 * c;
              float y[2] = {0.f, 0.f};
              for (int r = 0; r < groups; r += 2) {              // two or more
                y[0] += row[r * dv];
                y[1] += row[(r + 1) * dv];
              }
              o[x][c] = y[0] + y[1];
            }
            ss = fmaf(o[x][c], o[x][c], ss);
          }
          inv[x] = p.z ? rsqrtf(warp_sum(ss) / (float)dv + kRmsEps) : 1.f;
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int t = warp + 8 * x;
          T* orow = (T*)p.out + (t0 + t) * p.ldo + (long long)h * dv + lane;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (t >= n || lane + 32 * c >= dv) continue;
            float y = o[x][c];
            if (p.z) y = y * inv[x] * wt[c] * silu_f(z[x][c]);
            orow[32 * c] = Elem<T>::from_f(y);
          }
        }
      }
    }
    if (kSum) {
      float* dst = p.wsS + (size_t)blockIdx.x * hs;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) dst[(size_t)(r0 + r) * dv + j] = S[r];
      if (tid == 0) {
        p.wsA[blockIdx.x] = total;
        p.chains[blockIdx.x] = chain_of<kSimtBatch>(p, rg, g, blockIdx.x);
      }
      return;
    }
    if (g.last && p.state_out) {
      float* dst = p.state_out + ((size_t)g.slot * p.H + h) * hs;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) dst[(size_t)(r0 + r) * dv + j] = S[r];
    }
  }
}

// ---------------------------------------------------------------------------
// One token of one sequence and head: S = a S + k^T v, o = scale q S, read and
// written once in fp32 (8 dk dv bytes, the floor of the call: about 96% of its
// bytes at dk = dv = 128).  A block of 256 threads per (row, head); thread tid
// has the four columns 4 (tid % (dv / 4)) and every (256 / (dv / 4))-th row,
// R float4 of the state, all loaded before the first is used.  Bound by memory
// with many rows (500 rows, 16 heads of 128: 165 us for the kernel by itself, 170 to
// 175 call behind call, 6.1 TB/s, 0.93 of a plain copy's rate), by start and end with
// 64 (28.7 us, 4.7 TB/s: two blocks resident per SM, so 1024 blocks are 3.5 waves),
// by latency and the launch with one (2.7 us in a graph).
constexpr int kStepThreads = 256;

template <typename T, int R>
__global__ void __launch_bounds__(kStepThreads) hla_step(const Params p) {
  __shared__ float ks[128], qs[128], red[kStepThreads * 4], osum[4];
  pdl_wait();
  pdl_trigger();
  const int n = blockIdx.x, h = blockIdx.y, hk = h / (p.H / p.Hk);
  const int dk = p.dk, dv = p.dv, tid = threadIdx.x;
  const long long slot = p.slots ? __ldg(p.slots + n) : n;
  if (slot < 0) return;
  if (slot >= p.nslots) {
    if (tid == 0) gtr_flag(kStatusBadSlot);
    return;
  }
  const int per_row = dv / 4, rows = kStepThreads / per_row;   // threads of a row; rows a pass
  const int c4 = tid % per_row * 4, r0 = tid / per_row;
  const size_t base = ((size_t)slot * p.H + h) * dk * dv;
  const float* Si = p.state_in + base + c4;
  float4 S[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = r0 + r * rows;
    if (row < dk) S[r] = *reinterpret_cast<const float4*>(Si + (size_t)row * dv);
  }
  if (tid < dk) ks[tid] = ld_f((const T*)p.k + n * p.ldk + (long long)hk * dk + tid);
  else if (tid >= 128 && tid < 128 + dk)
    qs[tid - 128] = ld_f((const T*)p.q + n * p.ldq + (long long)hk * dk + tid - 128) * p.scale;
  const T* vr = (const T*)p.v + n * p.ldv + (long long)h * dv + c4;
  const float v0 = ld_f(vr), v1 = ld_f(vr + 1), v2 = ld_f(vr + 2), v3 = ld_f(vr + 3);
  // S + (a - 1) S + k v for a near one, as in the prompt kernel above (500 rows: 169 us, 168 with a rounded a)
  const float l = load_decay(p, n, h);
  const bool near_one = l > -1.f;
  const float a = near_one ? expm1_small(l * kLn2) : exp2f(l);
  const uint64_t a2 = tc::f2pack(a, a), v01 = tc::f2pack(v0, v1), v23 = tc::f2pack(v2, v3), zero = tc::f2pack(0.f, 0.f);
  __syncthreads();
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float* So = p.state_out + base + c4;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = r0 + r * rows;
    if (row < dk) {
      const float k = ks[row], q = qs[row];
      float4 s = S[r];
      const uint64_t k2 = tc::f2pack(k, k), s01 = tc::f2pack(s.x, s.y), s23 = tc::f2pack(s.z, s.w);
      const float2 x = tc::f2unpack(tc::ffma2(a2, s01, tc::ffma2(k2, v01, near_one ? s01 : zero)));
      const float2 y = tc::f2unpack(tc::ffma2(a2, s23, tc::ffma2(k2, v23, near_one ? s23 : zero)));
      s = make_float4(x.x, x.y, y.x, y.y);
      *reinterpret_cast<float4*>(So + (size_t)row * dv) = s;
      o.x = fmaf(q, s.x, o.x); o.y = fmaf(q, s.y, o.y);
      o.z = fmaf(q, s.z, o.z); o.w = fmaf(q, s.w, o.w);
    }
  }
  *reinterpret_cast<float4*>(red + r0 * dv + c4) = o;
  __syncthreads();
  float y = 0.f;
  if (tid < dv) {
    const int live = min(rows, dk);
    for (int r = 0; r < live; ++r) y += red[r * dv + tid];
  }
  if (p.z) {
    const float s = warp_sum(y * y);
    if ((tid & 31) == 0 && tid < 128) osum[tid >> 5] = s;
    __syncthreads();
    if (tid < dv) {
      float ss = 0.f;
      for (int i = 0; i < (dv + 31) / 32; ++i) ss += osum[i];
      y = y * rsqrtf(ss / (float)dv + kRmsEps) * (p.w ? p.w[tid] : 1.f) *
          silu_f(ld_f((const T*)p.z + n * p.ldz + (long long)h * dv + tid));
    }
  }
  if (tid < dv) ((T*)p.out)[n * p.ldo + (long long)h * dv + tid] = Elem<T>::from_f(y);
}

}  // namespace hla
}  // namespace gtr
