"""The plan of the decay walks without a GPU: whatever segments a walk or a piece of its
contraction is cut into, the states it passes on fit the area that the workspace has for
them.  The plan's header is compiled by the host compiler; the launches use the same functions."""
import ctypes
import itertools
import os
import subprocess

import pytest
import torch

import chunkwise_linear_rnn_fwd_b200 as pkg
from chunkwise_linear_rnn_fwd_b200 import gla as G

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PLAN = r"""
#include "decay_plan.h"
using namespace gla;
// the most states that a walk (K whole, V) passes on, over its pieces, in bytes
static size_t walk(const gla_decay_desc *d, bool tc, int whole, int V, long lines) {
  size_t most = 0;
  for (int k0 = 0; k0 < whole; k0 += kDecayPiece) {
    const DecaySplit s = decay_split(d, tc, whole, k0, V, lines);
    const long n = (decay_max_len(d) + (tc ? decay_chunk_tc() : decay_chunk_cc(s.K)) - 1) /
                   (tc ? decay_chunk_tc() : decay_chunk_cc(s.K));
    // the segments cover the chunks, and none of them is empty
    if (s.P < 1 || s.P > kDecayMaxSegments || s.P * (long)s.L < n || (s.P - 1) * (long)s.L >= n) return (size_t)-1;
    if (s.bytes > most) most = s.bytes;
  }
  return most;
}
extern "C" void plan(const gla_decay_desc *d, int tc, int bwd, size_t *need, size_t *area, size_t *total) {
  const int dk = d->dk, dv = d->dv;
  const long a = decay_lines(d, dk), b = decay_lines(d, dv);
  *need = 0;
  if (!bwd) {
    *need = walk(d, tc, dk, dv, b);
  } else {
    const bool together = dv <= kDecayPiece;
    const size_t x = walk(d, tc, dv, dk, together ? 2 * a + b : a), y = walk(d, tc, dk, dv, together ? 2 * a + b : b);
    *need = x > y ? x : y;
  }
  *area = decay_states_bytes(d);
  *total = 256 + decay_states_areas(d, bwd) * *area + (bwd ? decay_acc_bytes(d) : 0);
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    from chunkwise_linear_rnn_fwd_b200 import build
    build.build()
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cc").write_text(PLAN)
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "chunkwise_linear_rnn_fwd_b200", "csrc"), str(d / "plan.cc"),
                    "-o", str(d / "plan.so")], check=True)
    f = ctypes.CDLL(str(d / "plan.so")).plan
    size = ctypes.POINTER(ctypes.c_size_t)
    f.argtypes, f.restype = [ctypes.POINTER(G.gla_decay_desc), ctypes.c_int, ctypes.c_int, size, size, size], None

    def run(desc, tc, bwd):
        n = [ctypes.c_size_t() for _ in range(3)]
        f(ctypes.byref(desc), tc, bwd, *(ctypes.byref(x) for x in n))
        return [x.value for x in n]
    return run


HEADS = [(1, 1), (1, 3), (5, 4), (20, 4), (25, 4), (37, 4), (38, 4), (74, 4), (64, 16)]
LENGTHS = [(1, 0), (64, 0), (65, 0), (100, 0), (127, 0), (128, 0), (300, 0), (2000, 0), (16384, 0), (3000, 70), (3000, 2900)]
WIDTHS = [(64, 64), (64, 320), (64, 257), (33, 300), (128, 256), (256, 320), (256, 512), (256, 576), (200, 1), (1, 4096)]


@pytest.mark.parametrize("dk,dv", WIDTHS)
def test_states_of_every_piece_fit_their_area(plan, dk, dv):
    lib = pkg.load()
    for (B, H), (T, max_len), segments in itertools.product(HEADS, LENGTHS, (0, 1, 3, 32)):
        d = G._decay_desc(B, H, T, max_len, dk, dv, torch.float32, segments=segments)
        for bwd in (0, 1):
            size = lib.gla_decay_workspace_size(ctypes.byref(d), bwd)
            for tc in (0, 1):
                need, area, total = plan(d, tc, bwd)
                assert total == size, (B, H, T, max_len, segments, bwd)
                assert need <= area, (B, H, T, max_len, segments, bwd, tc, need, area)


def test_a_narrow_last_piece_beside_its_partial_sums(plan):
    """20 x 4 heads, d_v = 320: pieces of 256 and 64 channels, 80 CTAs.  The states of the
    second piece lie ahead of the partial sums of the first, not over them."""
    for T in (100, 128):
        d = G._decay_desc(20, 4, T, 0, 64, 320, torch.float32)
        need, area, total = plan(d, 0, 1)
        assert need <= area and total == 256 + area + (20 * 4 * T * 64 * 4 + 255) // 256 * 256
