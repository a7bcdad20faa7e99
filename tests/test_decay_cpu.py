"""Decay attention without a GPU: the oracle against the gated oracle and against
differences, workspace sizes, and every refusal of the calls."""
import ctypes

import numpy as np
import pytest
import torch

import chunkwise_linear_rnn_fwd_b200 as pkg
from chunkwise_linear_rnn_fwd_b200 import gla as G
from oracle import decay as oracle
from tests.decay_cases import Batch

ARG, SHAPE, MIS, WS = -1, -2, -3, -4


@pytest.fixture(scope="module")
def lib():
    from chunkwise_linear_rnn_fwd_b200 import build
    build.build()
    return pkg.load()


def test_oracle_is_the_gated_recurrence_with_a_constant_gate(oracle_mod):
    b = Batch([37], 3, 8, 12, torch.float32, seed=1)
    q, k, v, do = (b.seq(n, 0) for n in ("q", "k", "v", "do"))
    ld, h0, dh = b.ld.double().numpy(), b.seq("h0", 0), b.seq("dh", 0)
    la = np.repeat(ld[None, :, None], 37, 2)
    o, S = oracle.fwd(q, k, v, ld, h0)
    ro, rS = oracle_mod.fwd(q[None], k[None], v[None], la, h0=h0[None], gate="scalar")
    np.testing.assert_allclose(o, ro[0], rtol=0, atol=1e-12)
    np.testing.assert_allclose(S, rS[0], rtol=0, atol=1e-12)
    mine = oracle.bwd(q, k, v, ld, do, h0, dh)
    ref = oracle_mod.bwd(q[None], k[None], v[None], la, do[None], h0=h0[None], dh_final=dh[None], gate="scalar")
    for x, y in zip(mine, (ref[0], ref[1], ref[2], ref[4])):
        np.testing.assert_allclose(x, y[0], rtol=0, atol=1e-12)


def test_oracle_gradients_against_differences():
    b = Batch([9], 2, 3, 4, torch.float32, seed=2)
    x = [b.seq(n, 0) for n in ("q", "k", "v")] + [b.seq("h0", 0)]
    ld, do, dh = b.ld.double().numpy(), b.seq("do", 0), b.seq("dh", 0)

    def loss(q, k, v, h):
        o, S = oracle.fwd(q, k, v, ld, h)
        return (o * do).sum() + (S * dh).sum()

    g = oracle.bwd(*x[:3], ld, do, x[3], dh)
    rng = np.random.default_rng(0)
    for i in range(4):
        u = rng.standard_normal(x[i].shape)
        hi, lo = (loss(*(a + s * u if j == i else a for j, a in enumerate(x))) for s in (1, -1))
        assert abs((hi - lo) / 2 - (g[i] * u).sum()) <= 1e-11 * (1 + abs(hi) + abs(lo))


def desc(**kw):
    a = dict(B=2, H=4, T=300, max_len=0, dk=64, dv=64, dtype=torch.bfloat16, slots0=2, slots1=2)
    a.update(kw)
    d = G._decay_desc(a["B"], a["H"], a["T"], a["max_len"], a["dk"], a["dv"], torch.bfloat16, a["slots0"], a["slots1"],
                      a.get("segments", 0))
    if "code" in kw:
        d.dtype = kw["code"]
    d.workspace, d.workspace_bytes = 1 << 20, 1 << 40
    return d


BAD_DESCS = [(dict(B=0), ARG), (dict(H=0), ARG), (dict(T=0), ARG), (dict(dk=0), ARG), (dict(dv=0), ARG),
             (dict(max_len=-1), ARG), (dict(max_len=301), ARG), (dict(segments=-1), ARG), (dict(code=7), ARG),
             (dict(dk=257), SHAPE), (dict(dv=4097), SHAPE), (dict(B=1 << 19), SHAPE), (dict(segments=33), SHAPE)]


@pytest.mark.parametrize("kw,code", BAD_DESCS)
def test_bad_descriptors(lib, kw, code):
    d = desc(**kw)
    v = ctypes.byref(G.gla_view(4096, 0, 64, 256))
    a = ctypes.c_void_p(4096)
    cu = a if d.max_len > 0 else None
    assert lib.gla_decay_workspace_size(ctypes.byref(d), 0) == 0
    assert lib.gla_decay_fwd(ctypes.byref(d), v, v, v, a, cu, None, None, v, None, None, None) == code
    assert lib.gla_decay_bwd(ctypes.byref(d), v, v, v, a, cu, None, v, None, v, v, v, None, None) == code
    if not {"T", "max_len", "segments"} & set(kw):  # the step uses none of these
        assert lib.gla_decay_step(ctypes.byref(d), v, v, v, a, a, None, v, None) == code


def test_bad_arguments_enqueue_nothing(lib):
    """Each of these is refused by the host; the addresses are never touched."""
    vw = lambda p=4096, sb=300 * 256, sh=64, st=256: ctypes.byref(G.gla_view(p, sb, sh, st))  # noqa: E731
    v, a, mis = vw(), ctypes.c_void_p(4096), ctypes.c_void_p(4098)

    def fwd(d, q=v, o=v, ld=a, cu=None, h0=None, i0=None, hT=None, i1=None):
        return lib.gla_decay_fwd(ctypes.byref(d), q, v, v, ld, cu, h0, i0, o, hT, i1, None)

    assert lib.gla_decay_fwd(None, v, v, v, a, None, None, None, v, None, None, None) == ARG
    assert fwd(desc(), q=None) == ARG and fwd(desc(), q=vw(0)) == ARG and fwd(desc(), o=vw(st=-1)) == ARG
    assert fwd(desc(), q=vw(4097)) == MIS
    for shared in (vw(sh=0), vw(st=0), vw(sb=0)):  # an output whose rows lie on one another
        assert fwd(desc(), o=shared) == ARG
    assert fwd(desc(), ld=None) == ARG and fwd(desc(), ld=mis) == MIS
    assert fwd(desc(), h0=a, i0=mis) == MIS and fwd(desc(), hT=a, i1=mis) == MIS
    assert fwd(desc(), cu=a) == ARG and fwd(desc(max_len=5)) == ARG       # cu_seqlens and max_len go together
    assert fwd(desc(max_len=5), cu=mis) == MIS
    assert fwd(desc(), i0=a) == ARG and fwd(desc(), i1=a) == ARG          # an index without its pool
    assert fwd(desc(slots0=0), h0=a, i0=a) == ARG and fwd(desc(slots1=0), hT=a, i1=a) == ARG
    assert fwd(desc(slots0=1), h0=a) == ARG and fwd(desc(slots1=1), hT=a) == ARG   # fewer entries than sequences
    assert fwd(desc(), h0=mis) == MIS and fwd(desc(), hT=mis) == MIS
    d = desc()
    d.workspace = None
    assert fwd(d) == ARG
    d.workspace = (1 << 20) + 8
    assert fwd(d) == MIS
    d.workspace, d.workspace_bytes = 1 << 20, 255
    assert fwd(d) == WS

    def bwd(d, do=v, dq=v, ld=a, dh=None, dh0=None):
        return lib.gla_decay_bwd(ctypes.byref(d), v, v, v, ld, None, None, do, dh, dq, v, v, dh0, None)

    assert bwd(desc(), do=None) == ARG and bwd(desc(), dq=vw(0)) == ARG and bwd(desc(), ld=None) == ARG and bwd(desc(), ld=mis) == MIS
    assert bwd(desc(), dq=vw(sh=0)) == ARG and bwd(desc(), dq=vw(st=0)) == ARG
    assert bwd(desc(), dh=mis) == MIS and bwd(desc(), dh0=mis) == MIS
    wide = desc(dv=512)
    wide.workspace_bytes = lib.gla_decay_workspace_size(ctypes.byref(wide), 0)
    assert bwd(wide) == WS  # the forward's workspace lacks the partial sums

    def step(d, q=v, ld=a, state=a, index=None):
        return lib.gla_decay_step(ctypes.byref(d), q, v, v, ld, state, index, v, None)

    assert lib.gla_decay_step(None, v, v, v, a, a, None, v, None) == ARG
    assert step(desc(), q=None) == ARG and step(desc(), ld=None) == ARG and step(desc(), state=None) == ARG
    assert step(desc(), ld=mis) == MIS and step(desc(), index=mis) == MIS
    assert step(desc(), state=mis) == MIS and step(desc(slots1=1)) == ARG and step(desc(slots1=0), index=a) == ARG


def test_workspace_size(lib):
    """The status word always; the states of a split sequence; the partial sums of a wide backward."""
    size = lambda for_bwd=0, **kw: lib.gla_decay_workspace_size(ctypes.byref(desc(**kw)), for_bwd)  # noqa: E731
    assert size(B=64, H=16) == 256 == size(1, B=64, H=16)
    assert size(B=1, H=1, T=4096) > 256
    assert size(1, B=1, H=1, T=4096) - 256 == 3 * (size(B=1, H=1, T=4096) - 256)  # three walks beside each other
    assert size(1, B=64, H=16, dv=512) == 256 + 64 * 300 * 16 * 64 * 4
    assert size(1, B=64, H=16, dv=512, max_len=40) == 256 + 300 * 16 * 64 * 4  # T rows in all
    for max_len in range(1, 2000, 37):  # a shorter bound never needs more
        assert size(B=1, H=1, T=2000, max_len=max_len) <= size(B=1, H=1, T=2000)
    with pytest.raises(pkg.GLAError):
        pkg.decay_workspace_size(1, 1, 10, 300, 64, torch.bfloat16)
    with pytest.raises(ValueError):
        pkg.decay_workspace_size(1, 1, 10, 64, 64, torch.float16)


def test_tensors_of_the_host_are_refused():
    x = torch.zeros(1, 2, 8, 16)
    with pytest.raises(ValueError):
        pkg.gla_decay_fwd(x, x, x, torch.zeros(2))
    with pytest.raises(ValueError):
        pkg.gla_decay_bwd(x, x, x, torch.zeros(2), x)
    with pytest.raises(ValueError):
        pkg.gla_decay_step(x[:, :, 0], x[:, :, 0], x[:, :, 0], torch.zeros(2), torch.zeros(1, 2, 16, 16))
