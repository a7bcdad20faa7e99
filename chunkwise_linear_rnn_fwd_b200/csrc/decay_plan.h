// decay_plan.h -- how the walks of decay attention are cut: the contraction into pieces, the
// sequences into segments, and the workspace that this takes.  Plain C++ that needs no CUDA: the
// sizes that gla_decay_workspace_size returns and the launches come from the same functions,
// and a test compares the two over a grid of sizes on the CPU.
#pragma once

#include <stddef.h>

#include "gla.h"

namespace gla {

constexpr int kDecayPiece = 256;  // channels of one contraction
constexpr int kDecayTileV = 64;   // columns of V per CTA
constexpr int kDecayMaxSegments = 32;

// tokens of a chunk: on tensor cores, and on CUDA cores for a piece of K channels
constexpr int decay_chunk_tc() { return 128; }
inline int decay_chunk_cc(int K) { return K <= 128 ? 64 : 32; }

// CTAs of the CUDA-core walk that run at once: two an SM fit up to 64 channels (gradients of
// 4 x 4 heads of 700 tokens of 64 x 64 in fp32: 66 us, 76 if split for one an SM).  Counted for
// the whole contraction, not for its last and perhaps narrow piece: all pieces of a walk share
// one area for their states.
inline int decay_ctas_cc(int whole) { return whole <= 64 ? 2 * 148 : 148; }

// CTAs of an unsplit walk
inline long decay_lines(const gla_decay_desc *d, int V) {
  return (long)d->B * d->H * ((V + kDecayTileV - 1) / kDecayTileV);
}

inline int decay_max_len(const gla_decay_desc *d) { return d->max_len ? d->max_len : d->T; }

// Segments per sequence and chunks per segment of a walk.  Splitting reads y and z twice and
// passes states through memory, so a walk is split only while it (or, in a backward, the
// three together) leaves SMs idle: one CTA a segment and 64 columns, one or two an SM.  On
// tensor cores a chunk of the first pass takes half the time of one of the second: two
// segments lose up to 128 channels (4 x 8 heads of 2048 tokens of 128 x 128: 44 us instead of
// 43) and win above (2 x 4 heads of 16384 of 256 x 512: 348 instead of 476), and segments of
// one chunk do not pay (4 heads of 1024 of 128 x 128: 23 us whole, 20 in four segments, 21 in
// eight).  On CUDA cores every split pays (3 x 4 heads of 700 tokens of 64 x 64 in fp32: 121 us
// whole, 30 by chunks).  All of these from captured graphs, with states read and written.
inline int decay_most_segments(const gla_decay_desc *d, int chunk, long lines, int min_chunks, int least, int ctas) {
  const int n = (decay_max_len(d) + chunk - 1) / chunk;
  long p = d->segments ? d->segments : ctas / lines;
  if (!d->segments && p > n / min_chunks) p = n / min_chunks;
  if (p > kDecayMaxSegments) p = kDecayMaxSegments;
  if (p > n) p = n;
  return p < 1 || (!d->segments && p < least) ? 1 : (int)p;
}

// The piece from channel k0 on of a contraction over `whole` channels with V outputs: its
// channels K, P segments of L chunks, and the bytes of states that it passes on.
struct DecaySplit {
  int K, P, L;
  size_t bytes;
};
// lines: CTAs of the unsplit walk, or of the three that run beside each other
inline DecaySplit decay_split(const gla_decay_desc *d, bool tc, int whole, int k0, int V, long lines) {
  DecaySplit s;
  s.K = whole - k0 < kDecayPiece ? whole - k0 : kDecayPiece;
  const int chunk = tc ? decay_chunk_tc() : decay_chunk_cc(s.K);
  const int p = tc ? decay_most_segments(d, chunk, lines, 2, s.K <= 128 ? 3 : 2, 148)
                   : decay_most_segments(d, chunk, lines, 1, 2, decay_ctas_cc(whole));
  const int n = (decay_max_len(d) + chunk - 1) / chunk;
  s.L = (n + p - 1) / p;
  s.P = (n + s.L - 1) / s.L;
  s.bytes = s.P > 1 ? (size_t)d->B * d->H * s.P * s.K * V * sizeof(float) : 0;
  return s;
}

inline size_t decay_align(size_t x) { return (x + 255) / 256 * 256; }

// Bytes for the states of one walk, whichever of a call's it is and whatever path it takes: no
// piece has more channels than the whole, chunks below 32 tokens, or more CTAs to share.
inline size_t decay_states_bytes(const gla_decay_desc *d) {
  const int a = decay_most_segments(d, 32, decay_lines(d, d->dk), 1, 2, decay_ctas_cc(d->dv));
  const int b = decay_most_segments(d, 32, decay_lines(d, d->dv), 1, 2, decay_ctas_cc(d->dk));
  const int most = a > b ? a : b;
  return most > 1 ? decay_align((size_t)d->B * d->H * most * d->dk * d->dv * sizeof(float)) : 0;
}

// partial outputs of a backward whose contraction over dv is taken in pieces
inline size_t decay_acc_bytes(const gla_decay_desc *d) {
  const size_t rows = d->max_len ? (size_t)d->T : (size_t)d->B * d->T;
  return d->dv > kDecayPiece ? decay_align(rows * d->H * d->dk * sizeof(float)) : 0;
}

// Areas for states: the three walks of a backward run together unless they need partial outputs.
inline int decay_states_areas(const gla_decay_desc *d, bool bwd) { return bwd && d->dv <= kDecayPiece ? 3 : 1; }

}  // namespace gla
