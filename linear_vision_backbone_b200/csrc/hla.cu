// hla.cu -- linear attention with one decay per head: the C ABI of
// gtr_hla_fwd (prompts) and gtr_hla_step (single tokens), their argument
// checks, the segment plan and the launches.  Kernels: hla_simt.cuh (fp32 CUDA
// cores), hla_common.cuh (the scan over segments).
#include <atomic>

#include "gtr_gla.h"
#include "hla_common.cuh"
#include "hla_simt.cuh"

namespace {

using namespace gtr;

constexpr int kMaxDevices = 64;

bool valid_head_dim(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

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

// Tokens per segment and what follows from it.
struct Plan {
  int L;               // tokens per segment
  int nslot;           // segment slots (grid of the kernels)
  long long entries;   // summaries
  size_t off_a, bytes; // workspace: summaries, then log-decays
};

// The plan without cu_seqlens knows every length (T / nseq); with it, only
// their sum.  Shorter segments spread a long sequence over more SMs; each
// costs the summary of its tokens a second time, so a call whose sequences
// and heads fill the GPU takes long ones: L is about the tokens an SM gets
// when the work is spread evenly.
void make_plan(int nseq, int T, int H, int dk, int dv, bool equal, int sms, Plan* p) {
  const long long per_sm = 4;                                // resident blocks
  long long L = ((long long)T * H + sms * per_sm - 1) / (sms * per_sm);
  L = (L + hla::kC - 1) / hla::kC * hla::kC;
  if (L < hla::kC) L = hla::kC;
  const long long longest = equal ? T / nseq : T;
  long long cap = (longest + hla::kC - 1) / hla::kC * hla::kC;   // one segment holds any sequence
  if (cap < hla::kC) cap = hla::kC;
  if (L > cap) L = cap;
  p->L = (int)(L < (1ll << 30) ? L : (1ll << 30));
  if (equal) {
    const long long m = (longest + p->L - 1) / p->L;
    p->nslot = (int)(nseq * (m > 1 ? m : 1));
    p->entries = m > 1 ? nseq * (m - 1) : 0;
  } else {
    p->nslot = T / p->L + nseq;
    p->entries = T > p->L ? T / p->L + 1 : 0;
  }
  p->off_a = (size_t)p->entries * H * dk * dv * sizeof(float);
  p->bytes = p->off_a + (size_t)p->entries * H * sizeof(float);
}

template <typename T, int ROWS>
int launch_simt_rows(const hla::Params& p, bool sum, cudaStream_t st) {
  const dim3 grid((unsigned)p.nslot, (unsigned)p.H);
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
      !aligned(a->workspace, 16) || !aligned(a->g, 4) || !aligned(a->rms_w, 4) || !aligned(a->slots, 4) ||
      !aligned(a->seen, 4) || !aligned(a->cu_seqlens, 4))
    return GTR_ERR_ALIGNMENT;
  if (a->state_in && a->state_out && a->state_in != a->state_out) {
    const uintptr_t n = (uintptr_t)a->nslots * a->H * a->dk * a->dv * sizeof(float);
    const uintptr_t x = (uintptr_t)a->state_in, y = (uintptr_t)a->state_out;
    if (x < y + n && y < x + n) return GTR_ERR_INVALID_ARG;
  }
  *p = hla::Params{a->q, a->k, a->v, a->g, a->outgate, a->rms_w, a->out, a->state_in, a->state_out, a->slots, a->seen,
                   a->cu_seqlens, nullptr, nullptr, ld[0], ld[1], ld[2], ld[3], ld[4], a->nseq, a->T, a->Hk, a->H,
                   a->dk, a->dv, a->nslots, a->g_per_head != 0, a->scale, 0, 0};
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
  make_plan(nseq, T, H, dk, dv, false, sms, &a);
  if (T % nseq != 0) return a.bytes;
  Plan b;
  make_plan(nseq, T, H, dk, dv, true, sms, &b);
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
  make_plan(p.nseq, p.T, p.H, p.dk, p.dv, !p.cu, sms, &pl);
  if (pl.bytes > 0 && !args->workspace) return GTR_ERR_INVALID_ARG;
  if (args->workspace_bytes < pl.bytes) return GTR_ERR_NO_MEMORY;
  p.L = pl.L;
  p.nslot = pl.nslot;
  p.wsS = (float*)args->workspace;
  p.wsA = (float*)((char*)args->workspace + pl.off_a);
  const cudaStream_t st = (cudaStream_t)stream;
  if (pl.entries > 0) {
    if (launch_prompt(p, args->dtype, true, st)) return GTR_ERR_CUDA;
    const unsigned eb = (unsigned)((p.dk * p.dv / 4 + hla::kScanThreads - 1) / hla::kScanThreads);
    if (launch_pdl(hla::hla_scan, dim3((unsigned)pl.entries, (unsigned)p.H, eb), dim3(hla::kScanThreads), 0, st, p))
      return GTR_ERR_CUDA;
  }
  return launch_prompt(p, args->dtype, false, st) ? GTR_ERR_CUDA : GTR_OK;
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
