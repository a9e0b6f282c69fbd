// hla_common.cuh -- what the kernels of the head-decay linear attention share:
// their parameters, the split of the work, the scan over its cuts, and the
// decay.
//
// The split.  Sequence n has nb_n = ceil(len_n / C) blocks of C tokens in each of
// its H heads; each (sequence, head) is a run of nb_n + 1 units, its blocks and
// one more for what starting and ending it costs (a part of a block's time: the
// state is read and written).  All units stand in one line, sequence by
// sequence, head by head, and each of J groups takes an even share of the B = H
// sum (nb_n + 1) units and the blocks among them.  Only the device knows the
// lengths, so every kernel finds its range from cu_seqlens by itself.  With `cut` a range may end inside a (sequence,
// head): the part before the cut then has a summary (the state it makes from
// zero, and its decay) in workspace entry j, which the scan turns into the state
// the next group starts from; there are J entries whatever the sizes.  Without,
// a group takes the (sequence, head)s whose first block is in its range, whole.
// With offsets that are not those of a valid cu_seqlens no group has a unit, and
// the device status says so: their sequences may overlap, and B pass 31 bits.
#pragma once
#include "common.cuh"

namespace gtr {
namespace hla {

constexpr int kC = 128;            // tokens per block of the tensor-core kernels
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kMinLog = -110.0f; // e^-110 is zero in fp32

// The cuts of a (sequence, head), at the group with its first block: the
// summaries from there on (0: no such cut), the head, the state row, and
// whether it starts from state_in.
struct Chain {
  int m, h, slot, start;
};

struct Params {
  const void* q; const void* k; const void* v; const float* g; const void* z; const float* w; void* out;
  const float* state_in; float* state_out; const int* slots; const int* seen; const int* cu;
  float* wsS;                      // [J][dk][dv]: summaries, then start states of the next group
  float* ws0;                      // [J][dk][dv]: initial states of cut (sequence, head)s, by their first group
  float* wsA;                      // [J]: the summaries' log2-decays
  Chain* chains;                   // [J]
  long long ldq, ldk, ldv, ldz, ldo;
  int nseq, T, Hk, H, dk, dv, nslots, g_per_head;
  int seq_len;                     // T / nseq, without cu
  float scale;
  int J, cut;
};

// Rows of sequence n, and its blocks of C tokens.
template <int C> __device__ __forceinline__ int seq_rows(const Params& p, int n, int& a) {
  int b;
  if (p.cu) {
    a = min(max(__ldg(p.cu + n), 0), p.T);
    b = min(max(__ldg(p.cu + n + 1), a), p.T);
  } else {
    a = n * p.seq_len;
    b = a + p.seq_len;
  }
  return b - a;
}
__device__ __forceinline__ int n_blocks(int len, int C) { return len <= 0 ? 0 : (len - 1) / C + 1; }
// Units of the line of blocks that a (sequence, head) of this length takes.
__device__ __forceinline__ int n_units(int len, int C) { return n_blocks(len, C) + 1; }

// A place in the line: unit b of head h of sequence n.
struct Place {
  int n, h, b;
  // the place `off` units into sequence n of `per` units a head
  __device__ __forceinline__ void set(int seq, int off, int per) {
    n = seq;
    h = (unsigned)off / (unsigned)per;
    b = off - h * per;
  }
};

// Group j's range: the line's B units, the groups J that have any (at most one
// per unit), the places x0 and x1 it lies between and the sequences they fall
// into (nseq for x = B).
struct Range {
  int B, x0, x1, J;                // B < 2^31: the host refuses more
  int q, r;                        // B = q J + r: the first r groups have q + 1 units
  Place a, b;
  __device__ __forceinline__ int start(int j) const { return j >= J ? B : q * j + min(j, r); }
  __device__ __forceinline__ void set(int units, int groups, int j) {
    B = units;
    J = max(min(groups, units), 1);
    q = (unsigned)B / (unsigned)J;
    r = B - q * J;
    x0 = start(j);
    x1 = start(j + 1);
  }
};

// Units a head of sequence n by its offsets, or -1 where they are not those of a sequence.
template <int C> __device__ __forceinline__ int units_of(const Params& p, int n) {
  const int a = __ldg(p.cu + n), b = __ldg(p.cu + n + 1);
  return a < 0 || b < a || b > p.T ? -1 : n_units(b - a, C);
}

// By the whole block of threads.  `scratch`: 40 ints of shared memory, free
// again after the caller's next barrier.
template <int C> __device__ __forceinline__ void locate(const Params& p, int j, int* scratch, Range& g) {
  if (!p.cu) {
    const int nu = n_units(p.seq_len, C), per = nu * p.H;
    g.set(per * p.nseq, p.J, j);
    const int n0 = (unsigned)g.x0 / (unsigned)per, n1 = (unsigned)g.x1 / (unsigned)per;
    g.a.set(n0, g.x0 - n0 * per, nu);
    g.b.set(n1, g.x1 - n1 * per, nu);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  if (p.nseq <= 32) {
    // a lane for a sequence, every warp for itself: one load's latency and no barrier
    const int nu = lane < p.nseq ? units_of<C>(p, lane) : 0;
    const bool bad = __any_sync(0xffffffffu, nu < 0);
    int e = nu;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, e, d);
      if (lane >= d) e += o;
    }
    if (bad && tid == 0 && j == 0) gtr_flag(kStatusBadShape);
    g.set(bad ? 0 : __shfl_sync(0xffffffffu, e, 31) * p.H, p.J, j);
    const int s = (e - nu) * p.H;                                // this sequence's first unit
    auto at = [&](int x, Place& q) {
      if (x >= g.B) { q.set(p.nseq, 0, 1); return; }
      const int n = __popc(__ballot_sync(0xffffffffu, lane < p.nseq && s <= x)) - 1;
      q.set(n, x - __shfl_sync(0xffffffffu, s, n), __shfl_sync(0xffffffffu, nu, n));
    };
    at(g.x0, g.a);
    at(g.x1, g.b);
    return;
  }
  const int per = (p.nseq + blockDim.x - 1u) / blockDim.x;       // sequences per thread, consecutive ones
  const int n0 = min(tid * per, p.nseq), n1 = min(n0 + per, p.nseq);
  int mine = 0, bad = 0;
  for (int n = n0; n < n1; ++n) {
    const int nu = units_of<C>(p, n);
    mine += nu;
    bad |= nu < 0;
  }
  int inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) scratch[warp] = inc;
  if (tid == 0) {
    scratch[32] = p.nseq; scratch[33] = 0; scratch[34] = 1;
    scratch[35] = p.nseq; scratch[36] = 0; scratch[37] = 1;
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    if (tid == 0 && j == 0) gtr_flag(kStatusBadShape);
    g.set(0, p.J, j);
    g.a.set(p.nseq, 0, 1);
    g.b.set(p.nseq, 0, 1);
    return;
  }
  int before = inc - mine, total = 0;
  for (int w = 0; w < nw; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  g.set(total * p.H, p.J, j);
  for (int n = n0; n < n1; ++n) {
    const int nu = units_of<C>(p, n);
    const int s = before * p.H, e = (before + nu) * p.H;
    if (s <= g.x0 && g.x0 < e) { scratch[32] = n; scratch[33] = g.x0 - s; scratch[34] = nu; }
    if (s <= g.x1 && g.x1 < e) { scratch[35] = n; scratch[36] = g.x1 - s; scratch[37] = nu; }
    before += nu;
  }
  __syncthreads();
  g.a.set(scratch[32], scratch[33], scratch[34]);
  g.b.set(scratch[35], scratch[36], scratch[37]);
}

// A group's part of one (sequence, head).
struct Part {
  int n, h;
  int t0, len;        // its first token row, its tokens
  int nb;             // its blocks of C tokens (0: an empty sequence)
  bool first, last;   // it has the first / the last block of the (sequence, head)
  int slot;           // state row, or -1: the sequence is skipped
  bool start;         // the sequence starts from state_in
};

// Steps through a range of the line; every thread (or warp) of a group can
// walk it by itself and sees the same parts.  kFlag: of those that see a slot
// outside the pool, the one that records it.
struct Walk {
  Place at;
  int left;
};
template <int C, bool kFlag = false> __device__ __forceinline__ bool next_part(const Params& p, Walk& w, Part& g) {
  while (w.left > 0 && w.at.n < p.nseq) {
    int a;
    const int len = seq_rows<C>(p, w.at.n, a);
    const int nb = n_blocks(len, C);
    const int n = w.at.n, h = w.at.h, b0 = w.at.b;
    const int units = min(nb + 1 - b0, w.left);
    int end = min(b0 + units, nb);             // blocks b0 .. end - 1
    w.left -= units;
    w.at.b = 0;                                // what is left of the range starts the next head
    if (++w.at.h == p.H) { w.at.h = 0; w.at.n++; }
    if (b0 > 0) {
      if (!p.cut || b0 >= nb) continue;        // another group has it whole, or all of its blocks
    } else if (!p.cut) {
      end = nb;
    }
    g.n = n;
    g.h = h;
    g.first = b0 == 0;
    g.last = end == nb;
    g.t0 = a + b0 * C;
    g.len = min(len - b0 * C, (end - b0) * C);
    g.nb = end - b0;
    g.slot = p.slots ? __ldg(p.slots + n) : n;
    if (g.slot >= p.nslots && (p.state_in || p.state_out)) {
      if (kFlag) gtr_flag(kStatusBadSlot);
      g.slot = -1;
    }
    g.start = p.state_in && (!p.seen || __ldg(p.seen + n) > 0);
    if (g.slot >= 0) return true;
  }
  return false;
}

// The state a part of group j starts from, or null for zero.  A cut (sequence,
// head) has the scan's copy of its initial state: in place, the group of its
// end may write the state before the group of its start has read it.
__device__ __forceinline__ const float* start_state(const Params& p, const Part& g, int j) {
  const size_t hs = (size_t)p.dk * p.dv;
  if (!g.first) return p.wsS + (size_t)(j - 1) * hs;
  if (!g.start) return nullptr;
  if (!g.last) return p.ws0 + (size_t)j * hs;
  return p.state_in + ((size_t)g.slot * p.H + g.h) * hs;
}

// The part of a group before the cut at the end of its range; false when it
// ends with a (sequence, head).
template <int C> __device__ __forceinline__ bool cut_part(const Params& p, const Range& rg, Part& g) {
  const Place& b = rg.b;
  if (rg.x0 >= rg.x1 || b.n >= p.nseq) return false;
  int a;
  const int len = seq_rows<C>(p, b.n, a);
  const int h = b.h, e = b.b;                  // e units before the cut
  if (e == 0 || e >= n_blocks(len, C)) return false;   // nothing, or every block
  const int b0 = max(0, e - (rg.x1 - rg.x0));
  g.n = b.n;
  g.h = h;
  g.first = b0 == 0;
  g.last = false;
  g.t0 = a + b0 * C;
  g.len = (e - b0) * C;                        // whole blocks: the sequence goes on behind the cut
  g.nb = e - b0;
  g.slot = p.slots ? __ldg(p.slots + b.n) : b.n;
  if (g.slot >= p.nslots && (p.state_in || p.state_out)) g.slot = -1;
  g.start = p.state_in && (!p.seen || __ldg(p.seen + b.n) > 0);
  return g.slot >= 0;
}

// log2 of a decay: at most zero; below e^-110 nothing is left.  A NaN stays.
__device__ __forceinline__ float log2_decay(float g) {
  g = g > 0.f ? 0.f : g;
  g = g < kMinLog ? kMinLog : g;
  return g * kLog2e;
}
// e^x - 1 for -ln 2 < x <= 0 by its series to x^9 (what is left out is below x^10 / 10!, 2^-26 of the result) without a branch.
__device__ __forceinline__ float expm1_small(float x) {
  float y = 1.f / 362880.f;
  y = fmaf(y, x, 1.f / 40320.f);
  y = fmaf(y, x, 1.f / 5040.f);
  y = fmaf(y, x, 1.f / 720.f);
  y = fmaf(y, x, 1.f / 120.f);
  y = fmaf(y, x, 1.f / 24.f);
  y = fmaf(y, x, 1.f / 6.f);
  y = fmaf(y, x, 0.5f);
  return fmaf(y, x * x, x);
}
// Issued where it stands (a plain load may sink to its use, behind the wait it was to cover).
__device__ __forceinline__ float load_g(const Params& p, int t, int h) {
  float x;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(x) : "l"(p.g + (p.g_per_head ? (size_t)h : (size_t)t * p.H + h)));
  return x;
}
__device__ __forceinline__ float load_decay(const Params& p, int t, int h) { return log2_decay(load_g(p, t, h)); }

// The chain that starts at group j with cut part g.
template <int C> __device__ __forceinline__ Chain chain_of(const Params& p, const Range& rg, const Part& g, int j) {
  if (!g.first) return Chain{0, 0, 0, 0};
  // the summaries of this (sequence, head): of the groups that end before its blocks do
  int r, m = 1;
  const int end = rg.x1 - g.nb + n_blocks(seq_rows<C>(p, g.n, r), C);   // the unit behind them
  while (j + m < rg.J && rg.start(j + m + 1) < end) ++m;
  return Chain{m, g.h, g.slot, g.start};
}

// ---------------------------------------------------------------------------
// The states groups start from.  The group with the first block of a cut
// (sequence, head) walks its cuts: S = the initial state (copied to ws0), then
// entry i becomes S = e^{decay of part i} S + summary of part i.  One thread
// per four state elements and up to kScanAhead parts' loads in flight together.
// Bound by latency: a chain is a few thousand cycles whatever its width, so the
// grid (J, dk dv / 1024) is one wave of blocks, most of which have no chain and
// end at once (one element a thread: four waves, 16 us where this takes 8 with
// cold caches, dk = dv = 128, 74 groups).
constexpr int kScanThreads = 256;
constexpr int kScanAhead = 8;

__global__ void __launch_bounds__(kScanThreads) hla_scan(const Params p) {
  pdl_wait();
  pdl_trigger();
  const int j = blockIdx.x;
  const Chain ch = p.chains[j];
  if (ch.m == 0) return;
  const int per_state = p.dk * p.dv, e = (blockIdx.y * kScanThreads + threadIdx.x) * 4;
  if (e >= per_state) return;
  float* ws = p.wsS + (size_t)j * per_state + e;
  const float* wa = p.wsA + j;
  float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
  if (ch.start) {
    S = *reinterpret_cast<const float4*>(p.state_in + ((size_t)ch.slot * p.H + ch.h) * per_state + e);
    *reinterpret_cast<float4*>(p.ws0 + (size_t)j * per_state + e) = S;
  }
#pragma unroll 1
  for (int i0 = 0; i0 < ch.m; i0 += kScanAhead) {
    const int n = min(kScanAhead, ch.m - i0);
    float4 d[kScanAhead];
    float l[kScanAhead];
#pragma unroll
    for (int u = 0; u < kScanAhead; ++u)
      if (u < n) {
        d[u] = *reinterpret_cast<const float4*>(ws + (size_t)(i0 + u) * per_state);
        l[u] = wa[i0 + u];
      }
#pragma unroll
    for (int u = 0; u < kScanAhead; ++u)
      if (u < n) {
        const float f = exp2f(l[u]);
        S.x = fmaf(f, S.x, d[u].x); S.y = fmaf(f, S.y, d[u].y);
        S.z = fmaf(f, S.z, d[u].z); S.w = fmaf(f, S.w, d[u].w);
        *reinterpret_cast<float4*>(ws + (size_t)(i0 + u) * per_state) = S;
      }
  }
}

}  // namespace hla
}  // namespace gtr
