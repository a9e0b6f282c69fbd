// hla_common.cuh -- what the kernels of the head-decay linear attention share:
// their parameters, the split of packed sequences into segments and blocks of
// tokens, and the decay.
//
// A segment is a run of at most L consecutive tokens of one sequence (L a
// multiple of the block of kHlaC tokens).  Sequence n of start a and length
// len has ceil(len / L) segments, in slots a / L + n onwards; since
// floor((a + len) / L) + 1 >= floor(a / L) + ceil(len / L), the slots of
// different sequences are distinct and below T / L + nseq, so the grid is
// known without the lengths, which only the device has.  All but a sequence's
// last segment have a summary (the state the segment makes from zero, and its
// decay) in workspace entry a / L + i, distinct by the same argument and at
// most T / L.  Offsets that are not those of a valid cu_seqlens are clamped
// to [0, T], so no access leaves the tensors whatever it holds.
#pragma once
#include "common.cuh"

namespace gtr {
namespace hla {

constexpr int kC = 128;            // tokens per block of the tensor-core kernels; segments are multiples of it
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMinLog = -110.0f; // e^-110 is zero in fp32

struct Params {
  const void* q; const void* k; const void* v; const float* g; const void* z; const float* w; void* out;
  const float* state_in; float* state_out; const int* slots; const int* seen; const int* cu;
  float* wsS; float* wsA;          // segment summaries [entry][H][dk][dv], summed log2-decays [entry][H]
  float* ws0;                      // initial states of sequences of several segments [first entry][H][dk][dv]
  long long ldq, ldk, ldv, ldz, ldo;
  int nseq, T, Hk, H, dk, dv, nslots, g_per_head;
  float scale;
  int L;                           // tokens per segment
  int nslot;                       // segment slots, empty ones among them
};

// Segments sequence n of length len has.
__device__ __forceinline__ int n_segments(int len, int L) { return (int)(((long long)len + L - 1) / L); }

struct Segment {
  int n;          // sequence
  int t0, len;    // first token row, tokens
  int i, m;       // this segment of m
  int ws;         // workspace entry of the sequence's first segment
  long long slot; // state row, or -1: the sequence is skipped
  bool start;     // the sequence starts from state_in
};

// Rows of sequence n.
__device__ __forceinline__ void seq_rows(const Params& p, int n, int& a, int& b) {
  if (p.cu) {
    a = min(max(__ldg(p.cu + n), 0), p.T);
    b = min(max(__ldg(p.cu + n + 1), a), p.T);
  } else {
    const int len = p.T / p.nseq;
    a = n * len;
    b = a + len;
  }
}

// Segment slot s, by a whole warp; false for a slot that holds none.  Sequence
// n is the last one whose first slot a_n / L + n is <= s: these grow with n,
// so it is a count, 32 sequences a step.
__device__ __forceinline__ bool find_segment(const Params& p, int s, Segment& g) {
  const int lane = threadIdx.x & 31;
  int n;
  if (p.cu) {
    int count = 0;
    for (int n0 = 0; n0 < p.nseq; n0 += 32) {
      const int j = n0 + lane;
      bool le = false;
      if (j < p.nseq) le = min(max(__ldg(p.cu + j), 0), p.T) / p.L + j <= s;
      const int c = __popc(__ballot_sync(0xffffffffu, le));
      count += c;
      if (c < 32) break;
    }
    if (count == 0) return false;
    n = count - 1;
    int a, b;
    seq_rows(p, n, a, b);
    g.i = s - (a / p.L + n);
    g.ws = a / p.L;
    g.t0 = a;
    g.len = b - a;
    g.m = n_segments(g.len, p.L);
    if (g.i < 0 || g.i >= max(g.m, 1)) return false;   // a sequence of length zero has a slot for its state
  } else {
    const int len = p.T / p.nseq;
    g.m = max(1, n_segments(len, p.L));
    n = s / g.m;
    if (n >= p.nseq) return false;
    g.i = s - n * g.m;
    g.ws = n * (g.m - 1);
    g.t0 = n * len;
    g.len = len;
  }
  g.n = n;
  const int off = g.i * p.L;
  g.t0 += off;
  g.len = min(p.L, g.len - off);
  g.slot = p.slots ? __ldg(p.slots + n) : n;
  if (g.slot >= p.nslots && (p.state_in || p.state_out)) {
    if (lane == 0) gtr_flag(kStatusBadSlot);
    g.slot = -1;
  }
  g.start = p.state_in && (!p.seen || __ldg(p.seen + n) > 0);
  return g.slot >= 0;
}

// The state a segment starts from, or null for zero.  A sequence of several
// segments has the scan's copy of its initial state: in place, its last
// segment may write the state before its first one has read it.
__device__ __forceinline__ const float* start_state(const Params& p, const Segment& g, int h) {
  const size_t hs = (size_t)p.dk * p.dv;
  if (g.i > 0) return p.wsS + ((size_t)(g.ws + g.i - 1) * p.H + h) * hs;
  if (!g.start) return nullptr;
  if (g.m > 1) return p.ws0 + ((size_t)g.ws * p.H + h) * hs;
  return p.state_in + ((size_t)g.slot * p.H + h) * hs;
}

// log2 of a decay: at most zero; below e^-110 nothing is left.  A NaN stays.
__device__ __forceinline__ float log2_decay(float g) {
  g = g > 0.f ? 0.f : g;
  g = g < kMinLog ? kMinLog : g;
  return g * kLog2e;
}
__device__ __forceinline__ float load_decay(const Params& p, int t, int h) {
  return log2_decay(__ldg(p.g + (p.g_per_head ? (size_t)h : (size_t)t * p.H + h)));
}

// ---------------------------------------------------------------------------
// The states segments start from: for each sequence of several segments,
// S = its initial state, then entry i (the summary of segment i) is replaced by
// S = e^{decay of segment i} S + summary, the state segment i + 1 starts from.
// One thread per four state elements; grid (entries, H, dk dv / 4 / 128), a
// block whose entry is not the first of a sequence ends at once.
constexpr int kScanThreads = 128;
constexpr int kScanAhead = 8;      // segments whose loads are in flight together

__global__ void __launch_bounds__(kScanThreads) hla_scan(const Params p) {
  pdl_wait();
  pdl_trigger();
  const int entry = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31;
  int n, a, b;
  if (p.cu) {
    // the last sequence with a_n / L <= entry
    int count = 0;
    for (int n0 = 0; n0 < p.nseq; n0 += 32) {
      const int j = n0 + lane;
      bool le = false;
      if (j < p.nseq) le = min(max(__ldg(p.cu + j), 0), p.T) / p.L <= entry;
      const int c = __popc(__ballot_sync(0xffffffffu, le));
      count += c;
      if (c < 32) break;
    }
    if (count == 0) return;
    n = count - 1;
    seq_rows(p, n, a, b);
    if (a / p.L != entry) return;
  } else {
    const int per = n_segments(p.T / p.nseq, p.L) - 1;
    if (per < 1 || entry % per != 0) return;
    n = entry / per;
    if (n >= p.nseq) return;
    seq_rows(p, n, a, b);
  }
  const int m = n_segments(b - a, p.L) - 1;      // summaries
  const long long slot = p.slots ? __ldg(p.slots + n) : n;
  if (m < 1 || slot < 0 || (slot >= p.nslots && (p.state_in || p.state_out))) return;
  const int per_state = p.dk * p.dv;
  const int e = (blockIdx.z * kScanThreads + threadIdx.x) * 4;
  if (e >= per_state) return;
  float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p.state_in && (!p.seen || __ldg(p.seen + n) > 0)) {
    S = *reinterpret_cast<const float4*>(p.state_in + ((size_t)slot * p.H + h) * per_state + e);
    *reinterpret_cast<float4*>(p.ws0 + ((size_t)entry * p.H + h) * per_state + e) = S;
  }
  const size_t step = (size_t)p.H * per_state;
  float* ws = p.wsS + ((size_t)entry * p.H + h) * per_state + e;
  const float* wa = p.wsA + (size_t)entry * p.H + h;
  for (int i0 = 0; i0 < m; i0 += kScanAhead) {
    float4 d[kScanAhead];
    float l[kScanAhead];
#pragma unroll
    for (int u = 0; u < kScanAhead; ++u)
      if (i0 + u < m) {
        d[u] = *reinterpret_cast<const float4*>(ws + (i0 + u) * step);
        l[u] = wa[(size_t)(i0 + u) * p.H];
      }
#pragma unroll
    for (int u = 0; u < kScanAhead; ++u)
      if (i0 + u < m) {
        const float f = exp2f(l[u]);
        S.x = fmaf(f, S.x, d[u].x); S.y = fmaf(f, S.y, d[u].y);
        S.z = fmaf(f, S.z, d[u].z); S.w = fmaf(f, S.w, d[u].w);
        *reinterpret_cast<float4*>(ws + (i0 + u) * step) = S;
      }
  }
}

}  // namespace hla
}  // namespace gtr
