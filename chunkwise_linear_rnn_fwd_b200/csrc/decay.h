// decay.h -- what the decay-attention translation units share: the arguments of one
// walk over a batch of sequences, and how a CTA finds its sequence and its states.
//
// A walk computes, for every sequence and head, with lambda = exp(log_decay[h]),
//     S_t = lambda S_{t-1} + y_t^T z_t ,     o_t = x_t S_t
// (x, y: K channels, z, o: V channels).  The forward is one walk with (q, k, v).  The
// backward is three: with R_t = dL/dS_t = lambda R_{t+1} + q_t^T do_t,
//     dq_t = do_t S_t^T  (a walk over (do, v, k): the state is S^T),
//     dk_t = v_t R_t^T , dv_t = k_t R_t ,  dL/dS_0 = lambda R_1,
// the last two walks running from a sequence's last token to its first.
#pragma once

#include <cuda_bf16.h>

#include "internal.h"

namespace gla {

struct DView {
  void *p;
  long sb, sh, st;  // elements between sequences, heads, tokens
};

// fp32 states: entry e, head h, element (row k, column v) at
// e * slot + h * head + k * row + v * col
struct DPool {
  float *p;
  const int *idx;
  int slots;
  long slot, head, row, col;
};

struct DecayWalk {
  int nseq, H, T, max_len, K, V;
  int packed, reverse;
  const float *ld;
  const int *cu;
  DView x, y, z, o;
  DPool s0, s1;
  int alias;    // s0 and s1 are one pool
  int P, L;     // segments of L chunks per sequence (P > 1: states passed through ws)
  float *ws;    // [nseq*H][P][K][V]: entry 0 a copy of the start state, entry s the state after segment s-1
  float *acc;   // [H][rows][V] partial outputs of a contraction taken in pieces (rows: nseq * T, or T packed)
  int acc_in, acc_out;  // add the partial outputs to this walk's; write them instead of o
  // Launches of one call overlap: one with `lead` (every pre-pass) lets the next start once
  // all its CTAs have, one with `join` (the walk) or `pre_join` (the pre-pass) is such a next
  // one, which then ends no sooner than the launch ahead of it.  The walk of a split call
  // waits for its pre-pass before it reads the segments' states; with `settled` all pre-passes
  // had ended when the walk ahead of it, which has `wait_first`, let it start.
  int stage;  // 1 the pre-pass of a split walk, 2 the walk, 3 both
  int lead, join, pre_join, wait_first, settled;
#ifdef __CUDACC__
  __host__ __device__ __forceinline__ bool follows() const { return join || wait_first || P > 1; }
#endif
  unsigned *status;
};

// The walk of one call on CUDA cores (decay.cu) and on tensor cores (decay_tc.cu).
int decay_walk_cc(const DecayWalk &w, int dtype, cudaStream_t st);
bool decay_tc_takes(const DecayWalk &w, int dtype);
int decay_walk_tc(const DecayWalk &w, cudaStream_t st);

#ifdef __CUDACC__
namespace dev {

// A sequence's first row, its length and its coordinate along sb.  Bounds that are not a
// part of [0, T] no longer than max_len make an empty sequence and are reported.
struct DSeq {
  long row0;
  int len, b;
};
__device__ __forceinline__ DSeq decay_seq(const DecayWalk &w, int b) {
  DSeq s{0, w.T, b};
  if (w.packed) {
    const int a = __ldg(w.cu + b), e = __ldg(w.cu + b + 1);
    s.b = 0;
    s.row0 = a;
    s.len = e - a;
    if (a < 0 || e < a || e > w.T || s.len > w.max_len) {
      s.row0 = 0;
      s.len = 0;
      if (threadIdx.x == 0 && w.status) atomicOr(w.status, (unsigned)ST_INDEX);
    }
  }
  return s;
}

// log lambda of a head: a value above zero, or NaN, is taken as zero and reported
__device__ __forceinline__ double decay_rate(float x, unsigned *status) {
  if (x <= 0.f) return (double)x;
  if (threadIdx.x == 0 && status) atomicOr(status, (unsigned)ST_GATE_RANGE);
  return 0.0;
}
// lambda^n, formed in 64 bits (n log lambda loses what matters for long spans in 32); lambda^0 = 1
__device__ __forceinline__ double decay_pow(double rate, long n) { return n == 0 ? 1.0 : exp(rate * (double)n); }

// The pool entries that sequence b reads (i0) and writes (i1), -1: none.  One entry is
// written by the first sequence that names it, and a sequence whose start state another one
// overwrites starts from zero; both are reported.  Every thread of the CTA calls it, or
// (WARP) every lane of a warp, each warp finding the answer for itself.
template <bool WARP = false>
__device__ __forceinline__ void decay_slots(const DPool &s0, const DPool &s1, bool alias, int nseq, int b,
                                            unsigned *status, int &i0, int &i1) {
  i0 = s0.p ? (s0.idx ? __ldg(s0.idx + b) : b) : -1;
  i1 = s1.p ? (s1.idx ? __ldg(s1.idx + b) : b) : -1;
  bool bad = false;
  if (i0 >= s0.slots) i0 = -1, bad = s0.p != nullptr;
  if (i1 >= s1.slots) i1 = -1, bad |= s1.p != nullptr;
  if (s1.idx || (alias && s0.idx)) {
    int dup = 0, hazard = 0;
    const int me = WARP ? (int)(threadIdx.x & 31) : (int)threadIdx.x, all = WARP ? 32 : (int)blockDim.x;
    for (int j = me; j < nseq; j += all) {
      const int wj = s1.idx ? __ldg(s1.idx + j) : j;
      dup |= j < b && wj == i1;
      hazard |= alias && j != b && wj == i0 && (i1 != i0 || j < b);
    }
    // a negative entry equals another negative one: not a use
    dup = dup && i1 >= 0;
    hazard = hazard && i0 >= 0;
    dup = WARP ? __any_sync(0xffffffffu, dup) : __syncthreads_or(dup);
    hazard = WARP ? __any_sync(0xffffffffu, hazard) : __syncthreads_or(hazard);
    if (dup) i1 = -1;
    if (hazard) i0 = -1;
    bad |= dup || hazard;
  }
  if (i0 < 0) i0 = -1;
  if (i1 < 0) i1 = -1;
  if (bad && (WARP ? (threadIdx.x & 31) == 0 : threadIdx.x == 0) && status) atomicOr(status, (unsigned)ST_INDEX);
}

}  // namespace dev
#endif

}  // namespace gla
