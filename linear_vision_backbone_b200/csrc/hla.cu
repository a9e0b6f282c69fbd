// hla.cu -- linear attention with one decay per head: the C ABI of
// gtr_hla_fwd (prompts) and gtr_hla_step (single tokens), their argument
// checks, the segment plan and the launches.  Kernels: hla_tc.cuh (tensor
// cores), hla_simt.cuh (fp32 CUDA cores), hla_common.cuh (the scan over
// segments).
#include <cuda.h>

#include <algorithm>
#include <atomic>

#include "gtr_gla.h"
#include "hla_common.cuh"
#include "hla_simt.cuh"
#include "hla_tc.cuh"

namespace {
constexpr int kMaxDevices = 64;
}

namespace gtr {
// Multiprocessors of the current device; also the residual norm's.
int device_sms(int* sms) {
  static std::atomic<int> count[kMaxDevices];
  int dev;
  if (cudaGetDevice(&dev) != cudaSuccess) return GTR_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return GTR_ERR_UNSUPPORTED;
  int n = count[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    count[dev].store(n, std::memory_order_relaxed);
  }
  *sms = n;
  return GTR_OK;
}
}  // namespace gtr

namespace {

using namespace gtr;

bool valid_head_dim(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// 16-bit types and head dims the tensor-core kernels take
bool tc_shape(int dk, int dv, int dtype) { return dtype != GTR_F32 && dk >= 64 && dv >= 64; }

// How the work is split (hla_common.cuh) and the workspace that takes.
struct Plan {
  int J, cut;
  size_t off_0, off_c, off_a, bytes; // workspace: summaries, initial states, chains, log-decays
};

// Cutting spreads a long sequence evenly over the SMs, and costs the summaries
// (k and v before the cuts are read a second time) and two more launches; whole
// (sequence, head)s need neither, but the longest one bounds the time.  In units
// of one block of tokens of the outputs kernel on an SM of its own, a summary's
// block costs about kSum and the two launches kExtra.  Whole and cut, gated, in us:
//   bf16, 6 heads of 64:   1 x 256 tokens 13.2 and 18.9, 1 x 1024 30.7 and 19.7,
//     8 x 1600 46 and 40, 24 x 1600 51 and 80
//   bf16, 16 heads of 128: 1 x 512 24.5 and 29.4, 1 x 4096 147 and 68,
//     8 x 1600 129 and 149
//   fp32, 6 heads of 64:   1 x 32 11.9 and 16.1, 1 x 64 20.1 and 16.0,
//     8 x 1600 422 and 218, 24 x 512 139 and 214
// Without cu_seqlens the choice costs 0.3 % over 65 such cases (3.5 % at most, 24 x
// 1600 with 4 fp32 heads of 128).  With cu_seqlens the longest sequence may have
// all the tokens, so it is taken to: sequences that turn out equal can take longer
// than whole (24 x 1600 above 80 us for 51, 8 x 256 24 for 14).  The CUDA-core
// kernel cuts for twice as many groups as SMs: 24 x 1600 with 4 heads of 128 takes
// 842 us, as many groups as SMs 1051, three times 927, four times 850, although one
// block of its outputs is resident per SM from dk = dv = 64 on (180 registers a
// thread and more) and the second follows it; with even shares rounded up, 8 x 1600
// takes 313 us for 291.  Whole, an SM gains nothing by a second group, and each gets
// a (sequence, head).
void make_plan(int nseq, int T, int H, int dk, int dv, int dtype, bool equal, int sms, Plan* p) {
  const bool tc = tc_shape(dk, dv, dtype);
  const double kSum = tc ? 0.35 : 0.5, kExtra = tc ? 4.0 : 3.0;
  const long long C = tc ? hla::kC : hla::kSimtBatch;
  const long long slots = tc ? sms / (dv / 64) : sms;
  const long long len = equal ? T / nseq : T, longest = (len + C - 1) / C;
  const long long B = H * (equal ? nseq * (longest + 1) : T / C + 2ll * nseq);   // units; at most, with cu_seqlens
  const long long items = (long long)nseq * H;
  const double share = tc ? (double)((B + slots - 1) / slots) : (double)B / (double)slots;
  const double whole = equal ? (double)((items + slots - 1) / slots) * (double)(longest + 1)
                             : std::max(share, (double)longest);
  p->cut = longest > 1 && whole > share * (1.0 + kSum) + kExtra;
  const long long most = tc ? slots : p->cut ? 2 * slots : 4 * slots;            // groups
  long long J;
  if (!p->cut) J = std::min(items, most);
  else if (tc) J = (B + (long long)share - 1) / (long long)share;                // even shares, fewer summaries
  else J = std::min(B, most);                                                    // shares that differ by a unit
  p->J = (int)J;
  const size_t state = (size_t)dk * dv * sizeof(float);
  p->off_0 = p->cut ? J * state : 0;
  p->off_c = 2 * p->off_0;
  p->off_a = p->off_c + (p->cut ? J * sizeof(hla::Chain) : 0);
  p->bytes = p->off_a + (p->cut ? J * sizeof(float) : 0);
}

// ---- tensor-core launches
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled() {
  static std::atomic<EncodeTiledFn> fn{nullptr};
  EncodeTiledFn f = fn.load();
  if (!f) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess && ptr) {
      f = (EncodeTiledFn)ptr;
      fn.store(f);
    } else {
      (void)cudaGetLastError();
    }
  }
  return f;
}
// [T][heads][d] 16-bit rows of pitch ld elements, as boxes of 128 tokens x 64
// columns of one head in the 128-byte swizzle; tokens past T read as zero.
int map_rows(CUtensorMap* map, int dtype, const void* base, int T, int heads, int d, long long ld) {
  const EncodeTiledFn enc = encode_tiled();
  if (!enc) return GTR_ERR_CUDA;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)T};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)ld * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)hla::kC};
  const cuuint32_t one[3] = {1, 1, 1};
  const CUresult r = enc(map, dtype == GTR_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                         const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? GTR_OK : GTR_ERR_CUDA;
}

template <typename T, int DK, bool kSum, bool kGated, bool kPair>
int launch_tc_kernel(const hla::Params& p, const hla::Maps& maps, int halves, cudaStream_t st) {
  constexpr int smem = hla::Layout<T, DK, kSum>::kSmem;
  const auto kern = hla::hla_tc<T, DK, kSum, kGated, kPair>;
  static std::atomic<bool> done[kMaxDevices];
  int dev;
  if (cudaGetDevice(&dev) != cudaSuccess) return GTR_ERR_CUDA;
  if (!done[dev].load(std::memory_order_relaxed)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return GTR_ERR_CUDA;
    done[dev].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.J * halves));
  cfg.blockDim = dim3(kSum ? hla::kSumThreads : hla::kTcThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kPair ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p, maps, halves) == cudaSuccess ? GTR_OK : GTR_ERR_CUDA;
}
template <typename T, int DK>
int launch_tc_dk(const hla::Params& p, const hla::Maps& maps, bool sum, cudaStream_t st) {
  const int halves = p.dv / 64;
  if (sum) return launch_tc_kernel<T, DK, true, false, false>(p, maps, halves, st);
  if (!p.z) return launch_tc_kernel<T, DK, false, false, false>(p, maps, halves, st);
  if (halves == 2) return launch_tc_kernel<T, DK, false, true, true>(p, maps, halves, st);
  return launch_tc_kernel<T, DK, false, true, false>(p, maps, halves, st);
}
int launch_tc(const hla::Params& p, const hla::Maps& maps, int dtype, bool sum, cudaStream_t st) {
  if (dtype == GTR_F16)
    return p.dk == 64 ? launch_tc_dk<__half, 64>(p, maps, sum, st) : launch_tc_dk<__half, 128>(p, maps, sum, st);
  return p.dk == 64 ? launch_tc_dk<__nv_bfloat16, 64>(p, maps, sum, st)
                    : launch_tc_dk<__nv_bfloat16, 128>(p, maps, sum, st);
}

template <typename T, int ROWS>
int launch_simt_rows(const hla::Params& p, bool sum, cudaStream_t st) {
  const dim3 grid((unsigned)p.J);
  const size_t smem = (size_t)hla::simt_smem_floats(p.dk, p.dv, sum) * sizeof(float);   // below 48 KB
  if (sum) return launch_pdl(hla::hla_simt<T, ROWS, true>, grid, dim3(hla::kSimtThreads), smem, st, p);
  return launch_pdl(hla::hla_simt<T, ROWS, false>, grid, dim3(hla::kSimtThreads), smem, st, p);
}
template <typename T>
int launch_simt(const hla::Params& p, bool sum, cudaStream_t st) {
  switch (p.dk * p.dv / hla::kSimtThreads) {
    case 1: return launch_simt_rows<T, 1>(p, sum, st);
    case 2: return launch_simt_rows<T, 2>(p, sum, st);
    case 4: return launch_simt_rows<T, 4>(p, sum, st);
    case 8: return launch_simt_rows<T, 8>(p, sum, st);
    case 16: return launch_simt_rows<T, 16>(p, sum, st);
    case 32: return launch_simt_rows<T, 32>(p, sum, st);
    default: return launch_simt_rows<T, 64>(p, sum, st);
  }
}
int launch_prompt(const hla::Params& p, int dtype, bool sum, cudaStream_t st) {
  if (dtype == GTR_F32) return launch_simt<float>(p, sum, st);
  if (dtype == GTR_F16) return launch_simt<__half>(p, sum, st);
  return launch_simt<__nv_bfloat16>(p, sum, st);
}

template <typename T>
int launch_step(const hla::Params& p, cudaStream_t st) {
  const dim3 grid((unsigned)p.T, (unsigned)p.H);
  const dim3 block(hla::kStepThreads);
  switch (p.dk * p.dv / (4 * hla::kStepThreads)) {
    case 0:
    case 1: return launch_pdl(hla::hla_step<T, 1>, grid, block, 0, st, p);
    case 2: return launch_pdl(hla::hla_step<T, 2>, grid, block, 0, st, p);
    case 4: return launch_pdl(hla::hla_step<T, 4>, grid, block, 0, st, p);
    case 8: return launch_pdl(hla::hla_step<T, 8>, grid, block, 0, st, p);
    default: return launch_pdl(hla::hla_step<T, 16>, grid, block, 0, st, p);
  }
}

// n rows of `width` bytes, `pitch` apart.
struct Rows {
  const void* p;
  long long pitch, width, n;
};
// Whether two sets of rows share a byte.  Column blocks of one buffer (the same
// pitch, each between the other's columns) do not; sets of different pitches
// count as sharing when the ranges they span do.
bool overlap(const Rows& a, const Rows& b) {
  if (!a.p || !b.p || a.n < 1 || b.n < 1) return false;
  const long long x = (long long)(uintptr_t)a.p, y = (long long)(uintptr_t)b.p;
  if (x >= y + (b.n - 1) * b.pitch + b.width || y >= x + (a.n - 1) * a.pitch + a.width) return false;
  if (a.pitch != b.pitch) return true;
  const long long d = ((y - x) % a.pitch + a.pitch) % a.pitch;   // b's columns behind a's
  return d < a.width || a.pitch - d < b.width;
}

// Checks shared by both forms; on GTR_OK with *empty false, `p` is filled but
// for the workspace and the plan.
int check_args(const gtr_hla_args* a, bool step, hla::Params* p, bool* empty) {
  *empty = true;
  if (!a) return GTR_ERR_INVALID_ARG;
  if (a->dtype < 0 || a->dtype > 2) return GTR_ERR_INVALID_ARG;
  if (a->nseq < 0 || a->T < 0 || a->H < 0 || a->Hk < 0 || a->nslots < 0) return GTR_ERR_INVALID_ARG;
  if (!valid_head_dim(a->dk) || !valid_head_dim(a->dv)) return GTR_ERR_UNSUPPORTED;
  if (a->nseq == 0 || a->H == 0 || (a->T == 0 && !a->state_out)) return GTR_OK;
  if (a->Hk == 0 || a->H % a->Hk != 0) return GTR_ERR_INVALID_ARG;
  if (a->H > 65535) return GTR_ERR_UNSUPPORTED;
  // blocks of at least 16 tokens of all sequences and heads are counted in 31 bits
  if (!step && ((long long)a->T / hla::kSimtBatch + 2ll * a->nseq) * a->H >= (1ll << 31)) return GTR_ERR_UNSUPPORTED;
  if (step ? (a->T != a->nseq || a->cu_seqlens || a->seen) : (!a->cu_seqlens && a->T % a->nseq != 0))
    return GTR_ERR_INVALID_ARG;
  if (a->T > 0 && (!a->q || !a->k || !a->v || !a->g || !a->out)) return GTR_ERR_INVALID_ARG;
  if (a->rms_w && !a->outgate) return GTR_ERR_INVALID_ARG;
  if (step && (!a->state_in || !a->state_out)) return GTR_ERR_INVALID_ARG;
  if ((a->state_in || a->state_out) && !a->slots && a->nslots < a->nseq) return GTR_ERR_INVALID_ARG;
  const int es = a->dtype == GTR_F32 ? 4 : 2;
  const long long ld[5] = {a->ldq ? a->ldq : (long long)a->Hk * a->dk, a->ldk ? a->ldk : (long long)a->Hk * a->dk,
                           a->ldv ? a->ldv : (long long)a->H * a->dv, a->ldz ? a->ldz : (long long)a->H * a->dv,
                           a->ldo ? a->ldo : (long long)a->H * a->dv};
  for (int i = 0; i < 5; ++i) {
    if (ld[i] < (i < 2 ? (long long)a->Hk * a->dk : (long long)a->H * a->dv)) return GTR_ERR_INVALID_ARG;
    if (ld[i] > (1ll << 36)) return GTR_ERR_INVALID_ARG;
    if (ld[i] * es % 16 != 0) return GTR_ERR_ALIGNMENT;
  }
  if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->outgate, 16) ||
      !aligned(a->out, 16) || !aligned(a->state_in, 16) || !aligned(a->state_out, 16) ||
      !aligned(a->workspace, 16) || !aligned(a->rms_w, 16) || !aligned(a->g, 4) || !aligned(a->slots, 4) ||
      !aligned(a->seen, 4) || !aligned(a->cu_seqlens, 4))
    return GTR_ERR_ALIGNMENT;
  if (a->state_in && a->state_out && a->state_in != a->state_out) {
    const uintptr_t n = (uintptr_t)a->nslots * a->H * a->dk * a->dv * sizeof(float);
    const uintptr_t x = (uintptr_t)a->state_in, y = (uintptr_t)a->state_out;
    if (x < y + n && y < x + n) return GTR_ERR_INVALID_ARG;
  }
  // what is written shares nothing with what is read, but for states in place
  const long long st = (long long)a->H * a->dk * a->dv * (long long)sizeof(float);
  const Rows out{a->out, ld[4] * es, (long long)a->H * a->dv * es, a->T}, states{a->state_out, st, st, a->nslots};
  const long long nw = a->workspace ? (long long)std::min<size_t>(a->workspace_bytes, 1ull << 46) : 0;
  const Rows in[10] = {{a->q, ld[0] * es, (long long)a->Hk * a->dk * es, a->T},
                       {a->k, ld[1] * es, (long long)a->Hk * a->dk * es, a->T},
                       {a->v, ld[2] * es, (long long)a->H * a->dv * es, a->T},
                       {a->outgate, ld[3] * es, (long long)a->H * a->dv * es, a->T},
                       {a->g, a->H * 4ll, a->H * 4ll, a->g_per_head ? 1 : a->T},
                       {a->rms_w, a->dv * 4ll, a->dv * 4ll, 1},
                       {a->slots, 4, 4, a->nseq},
                       {a->seen, 4, 4, a->nseq},
                       {a->cu_seqlens, 4, 4, a->nseq + 1ll},
                       {a->workspace, nw, nw, nw > 0}};
  for (const Rows& r : in)
    if (overlap(out, r) || overlap(states, r)) return GTR_ERR_INVALID_ARG;
  if (overlap(out, states) || overlap(out, Rows{a->state_in, st, st, a->nslots})) return GTR_ERR_INVALID_ARG;
  *p = hla::Params{a->q, a->k, a->v, a->g, a->outgate, a->rms_w, a->out, a->state_in, a->state_out, a->slots, a->seen,
                   a->cu_seqlens, nullptr, nullptr, nullptr, nullptr, ld[0], ld[1], ld[2], ld[3], ld[4], a->nseq, a->T, a->Hk, a->H,
                   a->dk, a->dv, a->nslots, a->g_per_head != 0, a->T / a->nseq, a->scale, 0, 0};
  *empty = false;
  return GTR_OK;
}

}  // namespace

namespace gtr {
// The device status bits of this translation unit's kernels, cleared.  Part of
// gtr_last_device_status.
int hla_take_status(unsigned* bits) {
  const unsigned zero = 0;
  if (cudaMemcpyFromSymbol(bits, g_gtr_status, sizeof(*bits)) != cudaSuccess) return GTR_ERR_CUDA;
  if (cudaMemcpyToSymbol(g_gtr_status, &zero, sizeof(zero)) != cudaSuccess) return GTR_ERR_CUDA;
  return GTR_OK;
}
}  // namespace gtr

extern "C" {

GTR_API size_t gtr_hla_workspace_bytes(int nseq, int T, int H, int dk, int dv, int dtype) {
  if (nseq < 0 || T < 0 || H < 0 || H > 65535 || dtype < 0 || dtype > 2 || !valid_head_dim(dk) || !valid_head_dim(dv))
    return (size_t)-1;
  if (nseq == 0 || T == 0 || H == 0) return 0;
  int sms;
  if (device_sms(&sms)) return (size_t)-1;
  Plan a;
  make_plan(nseq, T, H, dk, dv, dtype, false, sms, &a);
  if (T % nseq != 0) return a.bytes;
  Plan b;
  make_plan(nseq, T, H, dk, dv, dtype, true, sms, &b);
  return a.bytes > b.bytes ? a.bytes : b.bytes;
}

GTR_API gtr_status_t gtr_hla_fwd(const gtr_hla_args* args, void* stream) {
  hla::Params p;
  bool empty;
  if (int rc = check_args(args, false, &p, &empty)) return (gtr_status_t)rc;
  if (empty) return GTR_OK;
  int sms;
  if (int rc = device_sms(&sms)) return (gtr_status_t)rc;
  Plan pl;
  make_plan(p.nseq, p.T, p.H, p.dk, p.dv, args->dtype, !p.cu, sms, &pl);
  if (pl.bytes > 0 && !args->workspace) return GTR_ERR_INVALID_ARG;
  if (args->workspace_bytes < pl.bytes) return GTR_ERR_NO_MEMORY;
  p.J = pl.J;
  p.cut = pl.cut;
  p.wsS = (float*)args->workspace;
  p.ws0 = (float*)((char*)args->workspace + pl.off_0);
  p.wsA = (float*)((char*)args->workspace + pl.off_a);
  p.chains = (hla::Chain*)((char*)args->workspace + pl.off_c);
  const cudaStream_t st = (cudaStream_t)stream;
  // an empty call (T = 0) only copies states: no tensor to map
  const bool tc = tc_shape(p.dk, p.dv, args->dtype) && p.T > 0;
  hla::Maps maps;
  if (tc && (map_rows(&maps.q, args->dtype, p.q, p.T, p.Hk, p.dk, p.ldq) ||
             map_rows(&maps.k, args->dtype, p.k, p.T, p.Hk, p.dk, p.ldk) ||
             map_rows(&maps.v, args->dtype, p.v, p.T, p.H, p.dv, p.ldv) ||
             map_rows(&maps.z, args->dtype, p.z ? p.z : p.v, p.T, p.H, p.dv, p.z ? p.ldz : p.ldv) ||
             map_rows(&maps.o, args->dtype, p.out, p.T, p.H, p.dv, p.ldo)))
    return GTR_ERR_CUDA;
  const auto launch = [&](bool sum) {
    return tc ? launch_tc(p, maps, args->dtype, sum, st) : launch_prompt(p, args->dtype, sum, st);
  };
  if (pl.cut) {
    if (launch(true)) return GTR_ERR_CUDA;
    const dim3 grid((unsigned)p.J, (unsigned)((p.dk * p.dv / 4 + hla::kScanThreads - 1) / hla::kScanThreads));
    if (launch_pdl(hla::hla_scan, grid, dim3(hla::kScanThreads), 0, st, p)) return GTR_ERR_CUDA;
  }
  return launch(false) ? GTR_ERR_CUDA : GTR_OK;
}

GTR_API gtr_status_t gtr_hla_step(const gtr_hla_args* args, void* stream) {
  hla::Params p;
  bool empty;
  if (int rc = check_args(args, true, &p, &empty)) return (gtr_status_t)rc;
  if (empty || p.T == 0) return GTR_OK;
  const cudaStream_t st = (cudaStream_t)stream;
  int rc;
  if (args->dtype == GTR_F32) rc = launch_step<float>(p, st);
  else if (args->dtype == GTR_F16) rc = launch_step<__half>(p, st);
  else rc = launch_step<__nv_bfloat16>(p, st);
  return rc ? GTR_ERR_CUDA : GTR_OK;
}

}  // extern "C"
