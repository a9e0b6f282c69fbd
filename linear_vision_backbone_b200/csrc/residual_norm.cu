// residual_norm.cu -- the norms around a residual branch with its gate and
// scale, one pass over the rows (gtr_residual_norm).
//
//     r = y [/ sqrt(mean(y^2) + eps) * post_w] [* act(gate)]
//     x_out = x + alpha * res_scale * r
//     out = x_out / sqrt(mean(x_out^2) + eps) * pre_w
//
// Bytes bound it: x, y and gate are read once and x_out and out written once.
// A row is held in the registers of its group of threads from the first load
// to the last store, so the two means cost reductions and no second read; all
// of a thread's loads are issued before the first is used.
//
// Measured: 16384 rows of 384, fp32 stream, fp16 branch, pre-norm: 15 to 16.5 us,
// 4.6 to 5.1 TB/s (a warp's row takes 66 registers: three blocks per SM, 4.6 waves;
// its 48 vectors leave half of the lanes idle in the second); 8191 rows of 5120 bf16
// with a SiLU gate, a scale and both norms: 76 to 81 us on several machines, 5.2 to
// 5.5 TB/s, 0.79 to 0.84 of a plain copy's rate, and 0.86 with 18944 rows, 0.91
// without the scale (start and end of the launch; 0.6 of the issue slots are taken,
// so conversions and products are two elements to an instruction); 18944 rows of an
// fp32 stream without a gate run at a copy's rate from D = 2048 on; nine rows of
// 4096: 3.0 us in a graph (latency).  A resident grid that copies rows ahead into shared memory
// and keeps the weights in registers was 10 to 50 % slower at every size from D =
// 256 to 8192 (fewer warps to hide the arithmetic).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <type_traits>

#include "gtr_gla.h"
#include "common.cuh"
#include "tc_ptx.cuh"

namespace gtr {
int device_sms(int* sms);   // hla.cu: multiprocessors of the current device
}

namespace {

using namespace gtr;

constexpr int kMaxD = 16384;             // 1024 threads of 16 elements
constexpr int kRowWarps = 8;            // rows per block where a warp has a row

struct NormArgs {
  const void* x; void* x_out; const void* y; const float* post_w; const void* gate;
  const float* res_scale; const float* pre_w; void* out;
  unsigned N, gate_rows;                // a rows' group of the gate; N below 2^31
  int D, post_norm, act;
  float alpha, eps, inv_d;              // 1 / D
};

// Two 16-bit elements to and from fp32: one conversion, and no packing.
template <typename T> struct Two;
template <> struct Two<__half> {
  using t = __half2;
  static __device__ __forceinline__ float2 to_f(t x) { return __half22float2(x); }
  static __device__ __forceinline__ t from_f(float a, float b) { return __floats2half2_rn(a, b); }
};
template <> struct Two<__nv_bfloat16> {
  using t = __nv_bfloat162;
  static __device__ __forceinline__ float2 to_f(t x) { return __bfloat1622float2(x); }
  static __device__ __forceinline__ t from_f(float a, float b) { return __floats2bfloat162_rn(a, b); }
};

// sigmoid(z).  For an fp32 branch e / (1 + e) or 1 / (1 + e) with e = e^-|z|, good to the last bits of fp32 down to
// its smallest numbers.  For a 16-bit branch 1 / (1 + 2^(-z log2 e)) by two approximate instructions (2^-22 each): the
// rounding of z log2 e makes it |z| 2^-24 + 2^-21 relative, far below the branch's own rounding, and zero below 2^-126;
// 8191 gated rows of 5120 bf16 are bound by instruction issue and took 84 us with the longer form, 82 with this.
template <typename TY> __device__ __forceinline__ float sigmoid(float z) {
  if constexpr (sizeof(TY) == 4) {
    const float e = expf(-fabsf(z));
    return (z < 0.f ? e : 1.f) / (1.f + e);
  }
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}

// VEC consecutive elements as loaded (16-byte accesses for VEC = 8), and as fp32.
template <typename T, int VEC> struct Pack {
  static constexpr int kWords = VEC == 1 ? 1 : VEC * (int)sizeof(T) / 16;
  using Word = std::conditional_t<VEC == 1, T, uint4>;
  Word w[kWords];
  // read once: the caches are left to the weights
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __ldcs(reinterpret_cast<const Word*>(p) + i);
  }
  __device__ __forceinline__ void widen(float (&v)[VEC]) const {
    if constexpr (VEC > 1 && sizeof(T) == 2) {
      typename Two<T>::t e[VEC / 2];
      memcpy(e, w, sizeof(e));
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) {
        const float2 f = Two<T>::to_f(e[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    } else {
      T e[VEC];
      memcpy(e, w, sizeof(e));
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = Elem<T>::to_f(e[i]);
    }
  }
  static __device__ __forceinline__ void store(T* p, const float (&v)[VEC]) {
    Word o[kWords];
    if constexpr (VEC > 1 && sizeof(T) == 2) {
      typename Two<T>::t e[VEC / 2];
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) e[i] = Two<T>::from_f(v[2 * i], v[2 * i + 1]);
      memcpy(o, e, sizeof(e));
    } else {
      T e[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) e[i] = Elem<T>::from_f(v[i]);
      memcpy(o, e, sizeof(e));
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) reinterpret_cast<Word*>(p)[i] = o[i];
  }
};
// A weight vector: shared by every row, so it stays in the caches.
template <int VEC> __device__ __forceinline__ void load_w(const float* p, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    v[0] = __ldg(p);
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(p) + i);
      v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
    }
  }
}

// Elementwise on a vector in fp32, two elements to an instruction (the same
// roundings): y *= w; y += f x; the sum of squares on top of s.
template <int VEC> __device__ __forceinline__ void mul(float (&y)[VEC], const float (&w)[VEC]) {
  if constexpr (VEC == 1) {
    y[0] *= w[0];
  } else {
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      const float2 r = tc::f2unpack(tc::fmul2(tc::f2pack(y[e], y[e + 1]), tc::f2pack(w[e], w[e + 1])));
      y[e] = r.x;
      y[e + 1] = r.y;
    }
  }
}
template <int VEC> __device__ __forceinline__ void mul(float (&y)[VEC], float f) {
  float w[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) w[e] = f;
  mul(y, w);
}
template <int VEC> __device__ __forceinline__ void add_scaled(float (&y)[VEC], float f, const float (&x)[VEC]) {
  if constexpr (VEC == 1) {
    y[0] = fmaf(f, x[0], y[0]);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      const float2 r =
          tc::f2unpack(tc::ffma2(tc::f2pack(f, f), tc::f2pack(x[e], x[e + 1]), tc::f2pack(y[e], y[e + 1])));
      y[e] = r.x;
      y[e + 1] = r.y;
    }
  }
}
template <int VEC> __device__ __forceinline__ float squares(const float (&y)[VEC], float s) {
  if constexpr (VEC == 1) {
    return fmaf(y[0], y[0], s);
  } else {
    uint64_t r = tc::f2pack(s, 0.f);
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      const uint64_t v = tc::f2pack(y[e], y[e + 1]);
      r = tc::ffma2(v, v, r);
    }
    const float2 f = tc::f2unpack(r);
    return f.x + f.y;
  }
}

// Sum over the threads of a row: a warp (kWarpRow), or the whole block.
template <bool kWarpRow>
__device__ __forceinline__ float row_sum(float s, float* red) {
  s = warp_sum(s);
  if constexpr (!kWarpRow) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) red[warp] = s;
    __syncthreads();
    s = warp_sum(lane < nw ? red[lane] : 0.f);
  }
  return s;
}

// kV vectors of VEC elements per thread; vector j of a row is thread j % G's.
template <typename TX, typename TY, int VEC, int kV, bool kWarpRow, int kMaxThreads, int kMinBlocks = 1>
__global__ void __launch_bounds__(kMaxThreads, kMinBlocks) residual_norm_kernel(const NormArgs a) {
  __shared__ float red[2][32];
  const int G = kWarpRow ? 32 : (int)blockDim.x;
  const int t = kWarpRow ? (threadIdx.x & 31) : (int)threadIdx.x;
  const unsigned row = kWarpRow ? blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  pdl_wait();
  pdl_trigger();
  if (row >= a.N) return;                 // whole warps only where a block has several rows
  const int nv = a.D / VEC;
  const size_t at = (size_t)row * (unsigned)a.D;
  const TX* xr = (const TX*)a.x + at;
  const TY* yr = a.y ? (const TY*)a.y + at : nullptr;
  const TY* gr = nullptr;
  if (a.gate) gr = (const TY*)a.gate + (a.gate_rows == 1 ? at : (size_t)(row / a.gate_rows) * (unsigned)a.D);
  Pack<TX, VEC> xp[kV];
  Pack<TY, VEC> yp[kV], gp[kV];
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    const int u = t + j * G;
    if (u < nv) {
      xp[j].load(xr + (size_t)u * VEC);
      if (yr) yp[j].load(yr + (size_t)u * VEC);
      if (gr) gp[j].load(gr + (size_t)u * VEC);
    }
  }
  float inv = 1.f;
  if (a.post_norm) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < kV; ++j)
      if (t + j * G < nv) {
        float y[VEC];
        yp[j].widen(y);
        s = squares(y, s);
      }
    inv = rsqrtf(row_sum<kWarpRow>(s, red[0]) * a.inv_d + a.eps);
  }
  // x + alpha res_scale r, in fp32 until the pre-norm has used it
  float x[kV][VEC];
  float s = 0.f;
  TX* xo = (TX*)a.x_out + at;
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    const int u = t + j * G;
    if (u >= nv) continue;
    xp[j].widen(x[j]);
    if (yr) {
      float y[VEC], w[VEC];
      yp[j].widen(y);
      if (a.post_norm) {
        if (a.post_w) {
          load_w<VEC>(a.post_w + u * VEC, w);
          mul(w, inv);
          mul(y, w);
        } else {
          mul(y, inv);
        }
      }
      if (gr) {
        float z[VEC];
        gp[j].widen(z);
        // the kind is the same for all: asked once a vector
        if (a.act != GTR_GATE_MUL) {
          float sg[VEC];
#pragma unroll
          for (int e = 0; e < VEC; ++e) sg[e] = sigmoid<TY>(z[e]);
          mul(y, sg);
        }
        if (a.act != GTR_GATE_SIGMOID) mul(y, z);
      }
      if (a.res_scale) {
        load_w<VEC>(a.res_scale + u * VEC, w);
        mul(y, w);
      }
      add_scaled(x[j], a.alpha, y);
    }
    if (yr || a.x_out != a.x) Pack<TX, VEC>::store(xo + (size_t)u * VEC, x[j]);
    s = squares(x[j], s);
  }
  if (!a.out) return;
  inv = rsqrtf(row_sum<kWarpRow>(s, red[1]) * a.inv_d + a.eps);
  TY* orow = (TY*)a.out + at;
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    const int u = t + j * G;
    if (u >= nv) continue;
    mul(x[j], inv);
    if (a.pre_w) {
      float w[VEC];
      load_w<VEC>(a.pre_w + u * VEC, w);
      mul(x[j], w);
    }
    Pack<TY, VEC>::store(orow + (size_t)u * VEC, x[j]);
  }
}

template <typename TX, typename TY, int VEC, int kV>
int launch_warp(const NormArgs& a, cudaStream_t st) {
  const unsigned blocks = (a.N + kRowWarps - 1) / kRowWarps;
  return launch_pdl(residual_norm_kernel<TX, TY, VEC, kV, true, 32 * kRowWarps>, dim3(blocks), dim3(32 * kRowWarps), 0,
                    st, a);
}
template <typename TX, typename TY, int VEC, int kV, int kMaxThreads, int kMinBlocks = 1>
int launch_block(const NormArgs& a, int threads, cudaStream_t st) {
  return launch_pdl(residual_norm_kernel<TX, TY, VEC, kV, false, kMaxThreads, kMinBlocks>, dim3(a.N),
                    dim3((unsigned)threads), 0, st, a);
}

int round32(int n) { return (n + 31) / 32 * 32; }

template <typename TX, typename TY>
int launch_typed(const NormArgs& a, bool vec, int sms, cudaStream_t st) {
  if (vec) {
    // A warp for a row of up to 64 vectors; else two vectors a thread, or one
    // while that leaves at most 512 threads a row and 1024 per SM in all. Gated
    // bf16, one and two: 888 rows of 1024 3.9 and 4.5 us, 1184 rows 4.9 and 5.0;
    // 592 rows of 2048 5.2 and 5.1, 1184 rows 7.8 and 7.0; 148 rows of 4096 3.8
    // and 4.3, 296 rows 5.5 and 5.5, 592 rows 8.7 and 7.4.
    const int nv = a.D / 8, threads = round32((nv + 1) / 2);
    if (nv <= 32) return launch_warp<TX, TY, 8, 1>(a, st);
    if (nv <= 64) return launch_warp<TX, TY, 8, 2>(a, st);
    if (nv <= 512 && (long long)a.N * nv < sms * 1024ll) return launch_block<TX, TY, 8, 1, 512>(a, round32(nv), st);
    // Four blocks of up to 320 threads per SM rather than three, at 48 registers: 18944 gated and scaled
    // rows of a 16-bit stream take 173 us for 195 at D = 5120 and 137 for 148 at 4096, but as long at 2048
    // (128 threads); more threads than 320 have no 48 registers for four blocks (6666 rows of 6144: 80 us,
    // 0.78 of a copy's rate; 5000 of 8192: 85, 0.73); an fp32 stream would spill and is at a copy's rate.
    if constexpr (sizeof(TX) == 2)
      if (threads > 128 && threads <= 320) return launch_block<TX, TY, 8, 2, 320, 4>(a, threads, st);
    if (threads <= 512) return launch_block<TX, TY, 8, 2, 512>(a, threads, st);
    return launch_block<TX, TY, 8, 2, 1024>(a, threads, st);
  }
  // one element an access: 8191 gated rows of 5119 bf16 take 247 us, of 5120 78
  if (a.D <= 256) return launch_warp<TX, TY, 1, 8>(a, st);
  if (a.D <= 4096) return launch_block<TX, TY, 1, 8, 512>(a, round32((a.D + 7) / 8), st);
  if (a.D <= 8192) return launch_block<TX, TY, 1, 16, 512>(a, round32((a.D + 15) / 16), st);
  return launch_block<TX, TY, 1, 16, 1024>(a, round32((a.D + 15) / 16), st);
}

bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// [p, p + n) and [q, q + m) share a byte
bool overlap(const void* p, size_t n, const void* q, size_t m) {
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return p && q && n && m && a < b + m && b < a + n;
}

}  // namespace

extern "C" GTR_API gtr_status_t gtr_residual_norm(const gtr_residual_norm_args* args, void* stream) {
  if (!args) return GTR_ERR_INVALID_ARG;
  const auto [x, x_out, y, post_w, gate, res_scale, pre_w, out, N, gate_rows, D, x_dtype, dtype, post_norm, gate_act,
              alpha, eps] = *args;
  if (x_dtype < 0 || x_dtype > 2 || dtype < 0 || dtype > 2) return GTR_ERR_INVALID_ARG;
  if (N < 0 || D < 0 || gate_act < GTR_GATE_MUL || gate_act > GTR_GATE_SILU) return GTR_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !(eps < 3.0e38f)) return GTR_ERR_INVALID_ARG;
  if (x_dtype != GTR_F32 && x_dtype != dtype) return GTR_ERR_UNSUPPORTED;
  if (D < 1 || D > kMaxD) return GTR_ERR_UNSUPPORTED;
  if (N > 0x7fffffffLL) return GTR_ERR_INVALID_ARG;
  if (N == 0) return GTR_OK;
  if (!x || !x_out) return GTR_ERR_INVALID_ARG;
  if (!y && (gate || post_norm || post_w || res_scale)) return GTR_ERR_INVALID_ARG;
  if (post_w && !post_norm) return GTR_ERR_INVALID_ARG;
  if (pre_w && !out) return GTR_ERR_INVALID_ARG;
  if (gate && (gate_rows < 1 || N % gate_rows != 0)) return GTR_ERR_INVALID_ARG;
  const size_t ex = x_dtype == GTR_F32 ? 4 : 2, ey = dtype == GTR_F32 ? 4 : 2;
  const size_t nx = (size_t)N * D * ex, ny = (size_t)N * D * ey, nw = (size_t)D * 4;
  const size_t ng = gate ? (size_t)(N / gate_rows) * D * ey : 0;
  if (!aligned(x, ex) || !aligned(x_out, ex) || !aligned(y, ey) || !aligned(gate, ey) || !aligned(out, ey) ||
      !aligned(post_w, 4) || !aligned(res_scale, 4) || !aligned(pre_w, 4))
    return GTR_ERR_ALIGNMENT;
  if ((x_out != x && overlap(x_out, nx, x, nx)) || overlap(x_out, nx, out, ny) || overlap(out, ny, x, nx))
    return GTR_ERR_INVALID_ARG;
  for (const void* w : {(const void*)x_out, (const void*)out}) {
    const size_t n = w == (const void*)x_out ? nx : ny;
    if (overlap(w, n, y, ny) || overlap(w, n, gate, ng) || overlap(w, n, post_w, nw) ||
        overlap(w, n, res_scale, nw) || overlap(w, n, pre_w, nw))
      return GTR_ERR_INVALID_ARG;
  }
  const bool vec = D % 8 == 0 && aligned(x, 16) && aligned(x_out, 16) && aligned(y, 16) && aligned(gate, 16) &&
                   aligned(out, 16) && aligned(post_w, 16) && aligned(res_scale, 16) && aligned(pre_w, 16);
  const NormArgs a{x, x_out, y, post_w, gate, res_scale, pre_w, out, (unsigned)N,
                   (unsigned)(gate ? gate_rows : 1), D, post_norm != 0, gate_act, alpha, eps, 1.0f / (float)D};
  const cudaStream_t st = (cudaStream_t)stream;
  int rc, sms;
  if ((rc = device_sms(&sms)) != 0) return (gtr_status_t)rc;
  if (x_dtype == GTR_F16) rc = launch_typed<__half, __half>(a, vec, sms, st);
  else if (x_dtype == GTR_BF16) rc = launch_typed<__nv_bfloat16, __nv_bfloat16>(a, vec, sms, st);
  else if (dtype == GTR_F32) rc = launch_typed<float, float>(a, vec, sms, st);
  else if (dtype == GTR_F16) rc = launch_typed<float, __half>(a, vec, sms, st);
  else rc = launch_typed<float, __nv_bfloat16>(a, vec, sms, st);
  return rc ? GTR_ERR_CUDA : GTR_OK;
}
